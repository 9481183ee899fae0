"""Host-side refusals of the norm / cache entry points (no call reaches a
kernel), and pins of the plain quantiser that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

import compressed_sparse_decode_gb300 as csd
import _records as R

P = C.c_void_p
FAKE = P(0x1000)


@pytest.fixture(scope="module")
def lib():
    csd.build()
    return csd.load()


def how(**kw):
    a = dict(norm=1, eps=1e-6, weight=None, rope_dim=64, rope_theta=10000.0)
    a.update(kw)
    return csd.csa_norm_rope(a["norm"], a["eps"], a["weight"], a["rope_dim"], a["rope_theta"])


BAD_HOW = [dict(eps=-1.0), dict(eps=float("nan")), dict(weight=0x1004), dict(norm=0, weight=0x1000),
           dict(rope_dim=-8), dict(rope_dim=20), dict(rope_theta=1.0), dict(rope_theta=float("inf"))]


@pytest.mark.parametrize("change, status", [
    (dict(x=None), 1), (dict(pos=None), 1), (dict(out=None), 1), (dict(x=P(0x1008)), 1), (dict(out=P(0x1004)), 1),
    (dict(dt=3), 1), (dict(dt=-1), 1), (dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1), (dict(D=0), 1),
    (dict(sb=-8), 1), (dict(st=12), 1), (dict(sh=4), 1), (dict(how=None), 1), (dict(status=P(0x1002)), 1),
    (dict(D=20), 2), (dict(D=520), 2), (dict(B=1 << 13, T=1 << 12), 2), (dict(B=1 << 12, T=1 << 12, H=128), 2),
] + [(dict(how=h), 1) for h in BAD_HOW])
def test_head_norm_rope_refuses(lib, change, status):
    a = dict(x=FAKE, dt=0, sb=65536, st=65536, sh=512, pos=FAKE, B=1, T=1, H=1, D=512, how={}, out=FAKE, status=None)
    a.update(change)
    h = None if a["how"] is None else C.byref(how(**a["how"]))
    args = [a["x"], a["dt"], a["sb"], a["st"], a["sh"], a["pos"], a["B"], a["T"], a["H"], a["D"], h, a["out"]]
    assert lib.csa_head_norm_rope(*args, a["status"], None) == status
    assert lib.csa_head_norm_rope_e4m3(*args, FAKE, a["status"], None) == status


def test_e4m3_form_needs_its_scale(lib):
    args = [FAKE, 0, 512, 512, 512, FAKE, 1, 1, 1, 512, C.byref(how()), FAKE]
    assert lib.csa_head_norm_rope_e4m3(*args, None, None, None) == csd.ERR_INVALID_ARG
    assert lib.csa_head_norm_rope_e4m3(*args, P(0x1008), None, None) == csd.ERR_INVALID_ARG


def desc(**kw):
    d = csd.csa_cache_desc()
    d.base, d.n_records, d.seq_stride, d.seq_capacity = 0x1000, 100, 50, 50
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("change, status", [
    (dict(cache=dict(base=None)), 1), (dict(cache=dict(base=0x1008)), 1), (dict(cache=dict(n_records=0)), 1),
    (dict(cache=dict(seq_capacity=0)), 1), (dict(cache=dict(seq_stride=40), B=2), 1),
    (dict(cache=dict(block_table=0x1000, page_records=0, max_pages=1)), 1),
    (dict(fmt=2), 1), (dict(first=None), 1), (dict(first=P(0x1004)), 1), (dict(count=P(0x1004)), 1), (dict(B=0), 1),
    (dict(T=0), 1), (dict(status=P(0x1001)), 1), (dict(B=1 << 13, T=1 << 12, cache=dict(seq_stride=64)), 2),
])
def test_cache_calls_refuse(lib, change, status):
    a = dict(cache={}, fmt=1, first=FAKE, count=None, B=1, T=1, status=None)
    a.update(change)
    d = desc(**a["cache"])
    assert lib.csa_cache_append(d, a["fmt"], 0, FAKE, 0, 512, 512, a["first"], a["count"], a["B"], a["T"], 1,
                                C.byref(how()), None, a["status"], None) == status
    assert lib.csa_cache_read(d, a["fmt"], 0, a["first"], a["count"], a["B"], a["T"], FAKE, a["status"],
                              None) == status


@pytest.mark.parametrize("change", [dict(x=None), dict(x=P(0x1002)), dict(dt=7), dict(sb=-8), dict(st=4),
                                    dict(pos_stride=0), dict(pos_stride=65537), dict(how=None),
                                    dict(how=dict(rope_dim=32)), dict(how=dict(rope_dim=128))]
                         + [dict(how=h) for h in BAD_HOW])
def test_append_refuses(lib, change):
    a = dict(x=FAKE, dt=0, sb=512, st=512, pos_stride=1, how={})
    a.update(change)
    h = None if a["how"] is None else C.byref(how(**a["how"]))
    assert lib.csa_cache_append(desc(), 0, 0, a["x"], a["dt"], a["sb"], a["st"], FAKE, None, 1, 1, a["pos_stride"], h,
                                None, None, None) == csd.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(key=None), dict(k_idx=None), dict(k_idx_scale=None), dict(key=0x1008),
                                    dict(k_idx=0x1004), dict(Ncap=0), dict(seq_stride=-8), dict(token_stride=4),
                                    dict(ring=1)])
def test_append_refuses_bad_index_keys(lib, change):
    a = dict(key=0x1000, seq_stride=128, token_stride=128, k_idx=0x1000, k_idx_scale=0x1000, Ncap=8, ring=0)
    a.update(change)
    i = csd.csa_index_append(a["key"], a["seq_stride"], a["token_stride"], a["k_idx"], a["k_idx_scale"], a["Ncap"])
    assert lib.csa_cache_append(desc(), 0, a["ring"], FAKE, 0, 512, 512, FAKE, None, 1, 1, 1, C.byref(how()),
                                C.byref(i), None, None) == csd.ERR_INVALID_ARG


def test_read_refuses_a_bad_output(lib):
    for out in (None, P(0x1008)):
        assert lib.csa_cache_read(desc(), 0, 0, FAKE, None, 1, 1, out, None, None) == csd.ERR_INVALID_ARG


def test_binding_refuses_host_tensors_and_wrong_formats():
    x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        csd.csa_head_norm_rope(x, torch.zeros((1, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="592"):
        csd.cache_desc(torch.zeros((4, 384), dtype=torch.uint8), 4)
    with pytest.raises(ValueError, match="384"):
        csd.cache_desc(torch.zeros((4, 592), dtype=torch.uint8), 4, fmt=csd.FORMAT_FP4)
    with pytest.raises(ValueError, match="format"):
        csd.cache_desc(torch.zeros((4, 592), dtype=torch.uint8), 4, fmt=5)
    d = desc()
    d._fmt = csd.FORMAT_FP4
    with pytest.raises(ValueError, match="592-byte"):
        csd._format(d, csd.FORMAT_FP8, "csa_decode_step")


def test_plain_quantiser_picks_nearest_values():
    """The reference quantiser against a brute-force nearest search and the
    format's own numbers."""
    rng = np.random.default_rng(0)
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(grid, R.E4M3)
    for v in np.concatenate([rng.standard_normal(200) * 3, R.E2M1, [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0]]):
        d = np.abs(np.abs(v) - R.E2M1)
        best = np.flatnonzero(d == d.min())
        want = best[0] if len(best) == 1 else [b for b in best if b % 2 == 0][0]
        assert R.nearest_code(v, R.E2M1) == want, v
    y = rng.standard_normal(512)
    codes, scales, E = R.fp4_record(y)
    assert np.abs(y[:448]).max() <= 2688 * 2.0 ** E < 2 * np.abs(y[:448]).max()
    rec = np.zeros((1, 384), np.uint8)
    rec[0, :224] = codes[0::2] | (codes[1::2] << 4)
    rec[0, 352:380], rec[0, 380] = scales, E + 127
    unit = np.repeat(R.E4M3[scales] * 2.0 ** E, 16)
    assert np.all(np.abs(R.fp4_values(rec)[0, :448] - y[:448]) <= unit)
    assert R.fp4_record(np.zeros(512))[2] == 0


def test_fp4_attention_refuses_like_the_fp8_calls(lib):
    """Same host checks and codes as the FP8 entry points, argument by argument."""
    good = desc(seq_stride=10, seq_capacity=10, n_records=10)
    over = desc(seq_stride=5, seq_capacity=10)
    E = csd.csa_attention_epilogue
    for c in [dict(q=None), dict(comp=csd.csa_cache_desc()), dict(comp=over, B=2), dict(W=600, R=600), dict(R=64),
              dict(scale=0.0), dict(k=4096), dict(T=129), dict(out=P(0x1008)), dict(status=P(0x1001)),
              dict(epi=E(1, 1.0, None, None)), dict(epi=E(0, 0.0, 0x2000, None)), dict(out=None), {}]:
        a = dict(q=FAKE, comp=good, R=128, W=128, B=1, T=1, k=4, out=FAKE, scale=0.1, status=None, epi=None)
        a.update(c)
        epi = None if a["epi"] is None else C.byref(a["epi"])
        head = (a["q"], FAKE, C.c_float(a["scale"]), a["comp"])
        tail = (a["out"], FAKE, epi, None, 0, a["status"], None)
        csa = (*head, FAKE, a["R"], a["W"], FAKE, FAKE, FAKE, a["B"], a["T"], a["k"], *tail)
        hca = (*head, FAKE, FAKE, a["R"], a["W"], FAKE, a["B"], a["T"], 128, *tail)
        # (with everything right and no workspace, a split row is refused for its workspace)
        want = lib.csa_sink_attention_decode_ex(*csa)
        assert lib.csa_sink_attention_decode_fp4(*csa) == want != csd.OK, c
        assert lib.hca_sink_attention_decode_fp4(*hca) == lib.hca_sink_attention_decode_ex(*hca) != csd.OK, c
    step = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, C.c_float(0.1), good, FAKE, 128, 128, FAKE, FAKE, 1, 1, 8, 4, 4,
            FAKE, FAKE, None, None, None, None, 0, None, None]
    assert lib.csa_decode_step_fp4(*step) == csd.ERR_WORKSPACE
    for i, bad, want in [(0, None, 1), (6, None, 1), (10, 64, 1), (19, P(0x1004), 1), (18, 9, 2)]:
        b = list(step)
        b[i] = bad
        assert lib.csa_decode_step_fp4(*b) == want, i
