"""The 8-bit cache calls refuse bad arguments before anything is launched
(fake device addresses are never touched), and the binding checks its tensors."""
import ctypes
import math

import numpy as np
import pytest

import _kv8 as R


@pytest.fixture(scope="module")
def dfl():
    import __graft_entry__ as g
    g.build()
    import block_diffusion_speculative_layer_gb300 as m
    m.lib()
    return m


P = ctypes.c_void_p
FAKE = P(0x1000)
GEOM = dict(codes=FAKE, exps=FAKE, n_pages=4, page=16, heads=8, hd=128, table=FAKE, pt_stride=8, start=FAKE, lens=FAKE,
            nseq=1, err=FAKE)
BAD_GEOM = [dict(codes=None), dict(exps=None), dict(table=None), dict(start=None), dict(lens=None), dict(n_pages=0),
            dict(page=8), dict(page=24), dict(page=1040), dict(heads=0), dict(hd=96), dict(hd=256), dict(pt_stride=0),
            dict(nseq=-1), dict(codes=P(0x1008)), dict(exps=P(0x1004)), dict(lens=P(0x1002)),
            dict(pt_stride=1 << 27), dict(n_pages=1 << 30)]


def write(dfl, **kw):
    a = dict(dict(GEOM, k=FAKE, v=FAKE, dtype=1, rows=16, ks=1024, vs=1024), **kw)
    return dfl.lib().df_op_kv8_write(a["k"], a["v"], a["dtype"], a["rows"], a["ks"], a["vs"], a["codes"], a["exps"],
                                     a["n_pages"], a["page"], a["heads"], a["hd"], a["table"], a["pt_stride"],
                                     a["start"], a["lens"], a["nseq"], a["err"], None)


def read(dfl, **kw):
    a = dict(dict(GEOM, k=FAKE, v=FAKE, dtype=1, rows=16), **kw)
    return dfl.lib().df_op_kv8_read(a["codes"], a["exps"], a["n_pages"], a["page"], a["heads"], a["hd"], a["table"],
                                    a["pt_stride"], a["start"], a["lens"], a["nseq"], a["rows"], a["dtype"], a["k"],
                                    a["v"], a["err"], None)


def attend(dfl, **kw):
    a = dict(dict(GEOM, q=FAKE, qs=4096, out=FAKE, os=4096, lse=FAKE, rows=16, hq=32, max_rows=16, max_len=100,
                  scale=0.1, causal=1, window=0, cla=0), **kw)
    return dfl.lib().df_op_attention_kv8(a["q"], a["qs"], a["out"], a["os"], a["lse"], a["rows"], a["hq"], a["codes"],
                                         a["exps"], a["n_pages"], a["page"], a["heads"], a["hd"], a["table"],
                                         a["pt_stride"], a["start"], a["lens"], a["nseq"], a["max_rows"],
                                         a["max_len"], a["scale"], a["causal"], a["window"], a["cla"], a["err"], None)


@pytest.mark.parametrize("call", [write, read, attend], ids=["write", "read", "attention"])
def test_bad_geometry(dfl, call):
    for bad in BAD_GEOM:
        assert call(dfl, **bad) == dfl.DF_EINVAL, bad
    assert call(dfl, rows=-1) == dfl.DF_EINVAL
    assert call(dfl, rows=0) == dfl.DF_OK      # nothing to do
    assert call(dfl, nseq=0) == dfl.DF_OK


def test_bad_rows_to_write_or_read(dfl):
    for call in (write, read):
        for bad in (dict(k=None), dict(v=None), dict(dtype=2), dict(dtype=-1), dict(k=P(0x1008))):
            assert call(dfl, **bad) == dfl.DF_EINVAL, bad
    for bad in (dict(ks=1016), dict(vs=8), dict(ks=1028), dict(vs=-1024), dict(dtype=0, ks=1026)):
        assert write(dfl, **bad) == dfl.DF_EINVAL, bad


def test_bad_attention(dfl):
    for bad in (dict(q=None), dict(out=None), dict(hq=36), dict(hq=4), dict(hq=0), dict(qs=4088), dict(os=4092),
                dict(qs=4100), dict(q=P(0x1008)), dict(out=P(0x1002)), dict(lse=P(0x1002)), dict(max_rows=-1),
                dict(max_len=-1), dict(causal=2), dict(window=-1), dict(window=5, causal=0), dict(scale=math.nan),
                dict(scale=math.inf), dict(cla=5), dict(cla=32), dict(cla=-1), dict(nseq=1 << 21)):
        assert attend(dfl, **bad) == dfl.DF_EINVAL, bad
    assert attend(dfl, max_rows=0) == dfl.DF_OK


def test_binding_wants_a_cuda_cache(dfl):
    torch = pytest.importorskip("torch")
    c = dfl.kv8_cache(3, 2, 64, 32, device="cpu")
    assert c.codes.shape == (3, 2, 2, 32, 64) and c.exps.shape == (3, 2, 32, 2)
    i = torch.zeros((1, 4), dtype=torch.int32)
    s, n = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros((1, 2, 64))
    for f in (lambda: dfl.kv8_write(c, x, x, i, s, n), lambda: dfl.kv8_read(c, i, s, n, 1),
              lambda: dfl.attention_kv8(x.view(1, 128).bfloat16(), c, i, s, n, 1, 1)):
        with pytest.raises(dfl.DfError):
            f()
    for bad in (dict(head_dim=96), dict(page_tokens=24), dict(page_tokens=0), dict(page_tokens=2048)):
        with pytest.raises(dfl.DfError):
            dfl.kv8_cache(**dict(dict(n_pages=2, n_kv_heads=1, device="cpu"), **bad))
    with pytest.raises(dfl.DfError):
        dfl.kv8_cache(0, 1, device="cpu")


def test_plain_form_rounds_as_torch_does():
    # the oracle's e4m3 rounding against torch's cast, ties and subnormals among the values
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(0)
    x = np.concatenate([R.STEPS, (R.STEPS[1:] + R.STEPS[:-1]) / 2, g.uniform(0, 448, 2000), 2.0 ** g.uniform(-12, 8, 999)])
    x = np.concatenate([x, -x])
    want = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    x = x.astype(np.float32).astype(np.float64)
    codes, e = R.quantise(np.stack([x, np.full_like(x, 448.0)], -1))
    assert (e == 127).all()
    np.testing.assert_array_equal(codes[:, 0], want)


def test_plain_exponents():
    e = lambda v: int(R.quantise(np.array([v, 0.0]))[1]) - 127
    assert e(448.0) == 0 and e(448.0001) == 1 and e(224.0) == -1 and e(1.75) == -8 and e(1.7500001) == -7
    assert e(0.0) == -100 and e(3e38) == 119 and e(1e-40) == -100
    codes, b = R.quantise(np.array([1.0, np.inf]))
    assert b == 255 and (codes == 0).all()


def test_attention_refuses_more_tiles_than_a_launch_counts(dfl):
    # 2^20 sequences of up to 2^20 rows and 8 heads of 4: far above 2^25 tiles
    for cla in (0, 12, 16):
        assert attend(dfl, nseq=1 << 20, rows=1 << 20, max_rows=1 << 20, cla=cla) == dfl.DF_EINVAL
