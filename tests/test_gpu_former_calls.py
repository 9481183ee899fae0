"""Calls over FP8 records that ran before the library had a second record format:
they take the same buffers and give the same results as ever."""
import math

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(512)


def fp8_step_bytes(csd, B, T, ncap, k):
    """Bytes of a step's workspace for FP8 records alone: logits, selection (twice
    B T k), top-k scratch, and for rows that are split over n CTA pairs (about one
    CTA an SM, at most one pair 64 candidates) their BF16 partials with (max, sum)."""
    def up(n):
        return -(-n // 256) * 256
    rows = B * T
    n = min(torch.cuda.get_device_properties(0).multi_processor_count // 2 // rows, -(-(k + 512) // 64))
    attention = up(rows * n * 128 * 512 * 2) + rows * n * 128 * 8 if n > 1 else 0
    return (up(4 * rows * ncap) + 2 * up(4 * rows * k) + up(csd.csa_workspace_bytes(csd.OP_TOPK, B, T, ncap, k))
            + up(attention))


# (24 rows: both formats split them alike, so that 4-bit records ask for more)
@pytest.mark.parametrize("wl", ["csa_b1_ctx1k_k64", "csa_b8_ctx16k32k_k512",
                                synth.Workload("b24_k300", "csa", B=24, T=1, ncap=1030, m=4, k=300, ctx=4100)],
                         ids=lambda w: getattr(w, "name", w))
def test_fp8_step_takes_a_workspace_for_fp8_records_alone(cuda_lib, wl):
    csd = cuda_lib
    x = synth.generate(wl, seed=3, device="cuda")
    wl = x.wl
    comp = csd.cache_desc(x.comp, wl.ncap, x.seq_stride, x.block_table, x.page_records)

    def step(ws):
        return csd.csa_decode_step(x.q_idx, x.q_idx_scale, x.w_idx, x.k_idx, x.k_idx_scale, x.q, x.sink, SCALE, comp,
                                   x.ring, wl.W, x.q_pos, x.n_comp, wl.m, wl.k, ws=ws)

    want = step(None)
    n = fp8_step_bytes(csd, wl.B, wl.T, wl.ncap, wl.k)
    assert n <= csd.csa_workspace_bytes(csd.OP_DECODE_STEP, wl.B, wl.T, wl.ncap, wl.k)
    buf = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    got = step(buf[:n])
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])
    assert torch.all(buf[n:] == 0xA5)
    with pytest.raises(csd.CsaError) as e:
        step(buf[:n - 1])
    assert e.value.status == csd.ERR_WORKSPACE
    assert csd.csa_read_device_error() == 0


def test_flat_buffer_of_fp8_records(cuda_lib):
    """A cache described by its bytes, by [B, pages, bytes of a page] and by [n, 592]
    is one cache."""
    csd = cuda_lib
    x = synth.generate("csa_b1_ctx1k_k64", seed=4, device="cuda")
    wl = x.wl
    idx = torch.arange(wl.k, dtype=torch.int32, device="cuda").view(1, 1, wl.k)
    cnt = torch.full((1, 1), wl.k, dtype=torch.int32, device="cuda")

    def out(records):
        comp = csd.cache_desc(records, wl.ncap, x.seq_stride)
        return csd.csa_sink_attention_decode(x.q, x.sink, SCALE, comp, x.ring, wl.W, idx, cnt, x.q_pos)[0]

    want = out(x.comp)
    for records in (x.comp.reshape(-1), x.comp.reshape(1, -1, 32 * 592)):
        assert torch.equal(out(records).view(torch.int16), want.view(torch.int16))
