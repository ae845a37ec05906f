"""Pins of the 8-bit form's oracle, and the library's host-side checks of the
8-bit entry points (CPU only: no compute call is made)."""
import numpy as np
import pytest

from oracle import q8_oracle as q8

torch = pytest.importorskip("torch")

import parameter_efficient_fine_gb300 as dora  # noqa: E402
from parameter_efficient_fine_gb300 import build as dbuild  # noqa: E402


def test_table_is_torchs():
    b = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    ref = b.view(torch.float8_e4m3fn).double().numpy()
    got = q8.e4m3_table()
    assert np.array_equal(np.isnan(ref), np.isnan(got))
    assert np.array_equal(ref[~np.isnan(ref)], got[~np.isnan(got)])


def test_hand_made_blocks():
    x = np.zeros((3, 130))
    x[0, :4] = [448.0, 1.0, -0.5, 447.0]        # scale 1
    x[0, 128:] = [449.0, 1.0]                   # past 448: scale 2, in a block of two columns
    x[1, :3] = [0.0, 1e-40, -0.0]               # below the smallest scale's range
    x[2, :4] = [np.nan, np.inf, -np.inf, 2.0]   # the scale comes from 2.0
    q, b = q8.q8_encode(x)
    assert b.tolist() == [[127, 128], [10, 10], [127 - 7, 10]]
    assert q[0, :4].tolist() == [0x7e, 0x38, 0xb0, 0x7e]
    assert q[0, 128:].tolist() == [0x76, 0x30]   # 224.5 -> 224, 0.5
    assert q[1, :3].tolist() == [0, 0, 0x80]
    assert q[2, :3].tolist() == [0x7f, 0x7f, 0x7f] and q8.q8_decode(q, b)[2, 3] == 2.0


def test_ties_go_to_even_and_match_torchs_cast():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((64, 256)).astype(np.float32)
    x[:, 0] = x[:, 128] = 448.0                 # scale 1 in every block
    x[:, 1:60] = (17 + 2 * np.arange(59)) * np.float32(0.5)      # midpoints of the E4M3 grid among them
    q, b = q8.q8_encode(x)
    assert (b == 127).all()
    assert np.array_equal(q, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("rows,cols,block_rows", [(5, 300, 1), (130, 140, 128), (256, 128, 128)])
def test_encode_is_the_identity_on_what_it_decodes_to(rows, cols, block_rows):
    x = np.random.default_rng(rows).standard_normal((rows, cols)) * 10.0
    q, b = q8.q8_encode(x, block_rows)
    v = q8.q8_decode(q, b, block_rows)
    assert np.abs(v - x).max() <= 2.0 ** -4 * np.abs(x).max()
    q2, b2 = q8.q8_encode(v, block_rows)
    assert np.array_equal(q8.q8_decode(q2, b2, block_rows), v)


def test_one_scale_per_tile_is_the_rows_largest():
    x = np.random.default_rng(0).standard_normal((256, 256))
    _, rowwise = q8.q8_encode(x, 1)
    _, tile = q8.q8_encode(x, 128)
    assert np.array_equal(tile, rowwise.reshape(2, 128, 2).max(1))


# ---- the library's argument checks -----------------------------------------
FAKE = 1 << 20   # a 256-byte aligned non-null address: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return dora.load_library()


def _caller(f, ok):
    def call(**kw):
        return f(*dict(ok, **kw).values())
    return call


def test_store_and_load_argument_errors(lib):
    store = _caller(lib.dora_q8_store, dict(act=1, x=FAKE, rows=4, cols=8, br=1, q=FAKE, sc=FAKE, stream=None))
    load = _caller(lib.dora_q8_load, dict(act=1, q=FAKE, sc=FAKE, rows=4, cols=8, br=1, x=FAKE, stream=None))
    for call in (store, load):
        assert call(act=5) == 4
        assert call(rows=-1) == 2 and call(cols=1 << 31) == 2 and call(br=2) == 2 and call(br=0) == 2
        assert call(rows=0) == 0 and call(cols=0) == 0
        assert call(x=None) == 1 and call(q=None) == 1 and call(sc=None) == 1
        assert call(x=FAKE + 1) == 3 and call(act=0, x=FAKE + 2) == 3


def test_compose_argument_errors(lib):
    fwd = _caller(lib.dora_compose_fwd_q8, dict(act=1, base=FAKE, lora=FAKE, g=FAKE, s=1.0, T=4, out=8, y=FAKE, q=FAKE,
                                                sc=FAKE, stream=None))
    assert fwd(act=9) == 4 and fwd(T=-1) == 2 and fwd(out=1 << 31) == 2
    assert fwd(T=0) == 0 and fwd(out=0) == 0
    for k in ("base", "lora", "g", "y", "q", "sc"):
        assert fwd(**{k: None}) == 1, k
    assert fwd(lora=FAKE + 1) == 3 and fwd(g=FAKE + 2) == 3
    bwd = _caller(lib.dora_compose_bwd_q8,
                  dict(act=1, dy=FAKE, q=FAKE, sc=FAKE, g=FAKE, norm=FAKE, s=1.0, T=64, out=64, db=FAKE, dl=FAKE,
                       dm=FAKE, ws=FAKE, wsb=1 << 30, stream=None))
    assert bwd(act=9) == 4 and bwd(T=-2) == 2 and bwd(out=0) == 0
    for k in ("dy", "q", "sc", "g", "norm", "db", "dl", "dm"):
        assert bwd(**{k: None}) == 1, k
    assert bwd(ws=None) == 5 and bwd(ws=FAKE + 64) == 5 and bwd(wsb=4) == 5
    assert bwd(db=FAKE + 1) == 3 and bwd(norm=FAKE + 2) == 3
    assert dora.dora_compose_bwd_q8_workspace(15360, 8192) >= 8192 * 4
    assert dora.dora_compose_bwd_q8_workspace(0, 8192) > 0 and dora.dora_compose_bwd_q8_workspace(-1, 8) == 0


def test_lora_grad_argument_errors(lib):
    f = _caller(lib.dora_lora_grad_q8, dict(dxa=FAKE, q=FAKE, sc=FAKE, T=64, inp=64, r=8, dA=FAKE, ws=FAKE,
                                            wsb=1 << 40, stream=None))
    assert f(T=-1) == 2 and f(inp=-16) == 2 and f(r=0) == 2 and f(r=1032) == 2
    assert f(inp=0) == 0
    for k in ("dxa", "q", "sc", "dA"):
        assert f(**{k: None}) == 1, k
    assert f(T=0, dA=None) == 1                   # T = 0 still writes dA (zeros)
    assert f(inp=72) == 3 and f(r=12) == 3 and f(q=FAKE + 8) == 3 and f(dxa=FAKE + 2) == 3 and f(dA=FAKE + 4) == 3
    assert f(ws=None) == 5 and f(ws=FAKE + 16) == 5 and f(wsb=16) == 5
    assert f(T=(1 << 31) - 1) == 2                # a tile past the last token has to be an int
    assert dora.dora_lora_grad_q8_workspace(64, 64, 0) == 0 and dora.dora_lora_grad_q8_workspace(64, 64, 8) > 0


@pytest.mark.parametrize("name", ["dora_matmul_q8", "dora_matmul_q8_t"])
def test_matmul_argument_errors(lib, name):
    f = _caller(getattr(lib, name), dict(q=FAKE, sc=FAKE, wq=FAKE, wsc=FAKE, T=64, out=64, inp=64, y=FAKE, ws=FAKE,
                                         wsb=1 << 40, stream=None))
    k, n = ("inp", "out") if name == "dora_matmul_q8" else ("out", "inp")
    assert f(T=-1) == 2 and f(**{k: 0}) == 2 and f(**{n: -16}) == 2 and f(**{n: 1 << 31}) == 2
    assert f(T=0) == 0 and f(**{n: 0}) == 0
    for a in ("q", "sc", "wq", "wsc", "y"):
        assert f(**{a: None}) == 1, a
    assert f(out=72) == 3 and f(inp=72) == 3 and f(q=FAKE + 8) == 3 and f(wq=FAKE + 8) == 3 and f(y=FAKE + 8) == 3
    assert getattr(dora, name + "_workspace")(64, 64, 64) == 0


def test_wrong_shapes_and_types_are_refused():
    u8 = torch.uint8
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, sc = torch.zeros(4, 256, dtype=u8), torch.zeros(4, 2, dtype=u8)
    with pytest.raises(ValueError, match="8-bit form"):
        dora.dora_q8_store(x, 1, q, torch.zeros(4, 1, dtype=u8), stream=0)
    with pytest.raises(ValueError, match="8-bit form"):
        dora.dora_q8_store(x, 128, q, sc, stream=0)
    with pytest.raises(TypeError, match="bytes"):
        dora.dora_q8_load(q, sc.float(), 1, x, stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        dora.dora_q8_store(x.t().contiguous().t(), 1, q, sc, stream=0)
    with pytest.raises(ValueError, match="CUDA tensors"):
        dora.dora_q8_store(x, 1, q, sc, stream=0)
    with pytest.raises(TypeError, match="not supported"):
        dora.dora_q8_store(x.half(), 1, q, sc, stream=0)
    g = torch.ones(256)
    with pytest.raises(ValueError, match="expected"):
        dora.dora_compose_fwd_q8(x, x.float(), g, 1.0, x, q, sc, stream=0)
    with pytest.raises(ValueError, match="expected"):
        dora.dora_compose_fwd_q8(x, x, g.bfloat16(), 1.0, x, q, sc, stream=0)
    w, wsc, ws = torch.zeros(128, 256, dtype=u8), torch.zeros(1, 2, dtype=u8), torch.zeros(256, dtype=u8)
    with pytest.raises(ValueError, match="expected"):
        dora.dora_matmul_q8(q, sc, w, wsc, torch.zeros(4, 256, dtype=torch.bfloat16), ws, stream=0)
    with pytest.raises(ValueError, match="8-bit form"):
        dora.dora_matmul_q8_t(q, sc, w, wsc, x, ws, stream=0)
    with pytest.raises(ValueError, match="expected"):
        dora.dora_lora_grad_q8(torch.zeros(4, 8), q, sc, torch.zeros(8, 256), ws, stream=0)


def test_ops_registered_and_fake_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode

    import parameter_efficient_fine_gb300.ops  # noqa: F401  (registers torch.ops.dora.*)

    bf, u8 = torch.bfloat16, torch.uint8
    with FakeTensorMode():
        x = torch.empty(8, 272, device="cuda", dtype=bf)
        q, sc = torch.ops.dora.q8_store(x, 1)
        assert q.shape == (8, 272) and sc.shape == (8, 3) and q.dtype == sc.dtype == u8
        wq, wsc = torch.ops.dora.q8_store(torch.empty(144, 272, device="cuda"), 128)
        assert wq.shape == (144, 272) and wsc.shape == (2, 3)
        assert torch.ops.dora.q8_load(q, sc, 1, torch.float32).dtype == torch.float32
        y = torch.ops.dora.matmul_q8(q, sc, wq, wsc)
        assert y.shape == (8, 144) and y.dtype == bf
        g = torch.empty(144, device="cuda")
        z, vq, vsc = torch.ops.dora.compose_q8(y, y, g, g, g, 1.0)
        assert z.shape == y.shape and vq.shape == y.shape and vsc.shape == (8, 2)
        db, dl, dm = torch.ops.dora.compose_bwd_q8(y, vq, vsc, g, g, 1.0)
        assert db.dtype == dl.dtype == bf and dm.shape == (144,) and dm.dtype == torch.float32
        assert torch.ops.dora.matmul_q8_t(vq, vsc, wq, wsc).shape == (8, 272)
        dA = torch.ops.dora.lora_grad_q8(torch.empty(8, 16, device="cuda", dtype=bf), q, sc)
        assert dA.shape == (16, 272) and dA.dtype == torch.float32
        A, B = torch.empty(16, 272, device="cuda"), torch.empty(144, 16, device="cuda")
        out = torch.ops.dora.linear_q8(x, wq, wsc, A, B, g, g, g, 1.0)
        assert out[0].shape == (8, 144) and out[0].dtype == bf and out[5].shape == (8, 16)
