"""What cache_desc takes and refuses, on host tensors that say they are on a GPU
(no call reaches the library)."""
import pytest
import torch

import compressed_sparse_decode_gb300 as csd


class OnGpu(torch.Tensor):
    """A host tensor that gives itself out as one on cuda:0."""
    is_cuda = True

    def get_device(self):
        return 0


class OnSecondGpu(OnGpu):
    def get_device(self):
        return 1


def on_gpu(shape, dtype=torch.uint8, cls=OnGpu):
    return torch.zeros(shape, dtype=dtype).as_subclass(cls)


@pytest.mark.parametrize("fmt", [csd.FORMAT_FP8, csd.FORMAT_FP4])
def test_records_of_any_dense_shape(fmt):
    size = csd.FORMAT_BYTES[fmt]
    for shape in ((24, size), (2, 12, size), (24 * size,), (2, 3, 4 * size), (2, 3, 4, size), (3, 4, 2 * size)):
        rec = on_gpu(shape)
        d = csd.cache_desc(rec, 12, seq_stride=12, fmt=fmt)
        assert (d.n_records, d.base, d._copied) == (24, rec.data_ptr(), False), shape


@pytest.mark.parametrize("fmt", [csd.FORMAT_FP8, csd.FORMAT_FP4])
def test_records_of_a_wrong_size(fmt):
    size, other = csd.FORMAT_BYTES[fmt], csd.FORMAT_BYTES[1 - fmt]
    # (37 * 384 = 24 * 592: whole records of either format, but marked as the other's)
    for shape in ((24, other), (37, 24, other), (24, 2 * size), (12, 2 * size), (24 * size + 16,), (2, 3, size + 1)):
        with pytest.raises(ValueError, match=str(size)):
            csd.cache_desc(on_gpu(shape), 12, seq_stride=12, fmt=fmt)


@pytest.mark.parametrize("fmt", [csd.FORMAT_FP8, csd.FORMAT_FP4])
def test_block_table_on_another_gpu_than_the_records(fmt):
    """The kernels read both on one device: a table elsewhere is never described."""
    rec = on_gpu((24, csd.FORMAT_BYTES[fmt]))
    for records, cls in ((rec, OnSecondGpu), (rec.as_subclass(OnSecondGpu), OnGpu)):
        table = on_gpu((2, 3), torch.int32, cls)
        with pytest.raises(ValueError, match="block_table is on cuda"):
            csd.cache_desc(records, 12, block_table=table, page_records=4, fmt=fmt)
    d = csd.cache_desc(rec, 12, block_table=on_gpu((2, 3), torch.int32), page_records=4, fmt=fmt)
    assert (d.max_pages, d._seqs, d._dev) == (3, 2, 0)
