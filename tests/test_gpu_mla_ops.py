"""The products around latent attention on the GPU against float64.

Tolerance: inputs are exact; a sum of K products in binary32 is off by at most
K 2^-23 of the sum of their magnitudes (the tensor cores may truncate, so a whole step
of each partial sum); the result is rounded to bf16, half a step being 2^-8 of it at most."""
import numpy as np
import pytest
import torch

from oracle import mla

pytestmark = pytest.mark.gpu

ROWS = [1, 3, 31, 32, 33, 127, 128, 129, 300]


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def padded(x, pad, fill=float("nan")):
    """Rows of x on the GPU with `pad` elements behind each."""
    x = x.flatten(1)
    wide = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=torch.bfloat16)
    wide[:, :x.shape[1]] = x
    return wide.cuda()


def f64(x):
    return x.double().numpy()


def outputs(rows, width, pad):
    """An output with rows behind the last and elements behind each row that must stay."""
    return torch.full((rows + 5, width + pad), 7.0, dtype=torch.bfloat16, device="cuda")


def run(op, rows, heads, pad=0, w_pad=0, seed=0, x=None, w=None, stream=None):
    import paged_quantized_kv_gqa_gb300 as pa
    K = 128 if op == "absorb" else 512
    w = randn(seed, heads, 256, 512, scale=K ** -0.5) if w is None else w
    wide = torch.full((heads, 256 * 512 + w_pad), float("nan"), dtype=torch.bfloat16)
    wide[:, :256 * 512] = w.flatten(1)
    wd = wide.cuda()
    shape = {"absorb": (rows, heads, 192), "project": (rows, heads, 512), "expand": (rows, 512)}[op]
    x = randn(seed + 1, *shape) if x is None else x
    xd = padded(x, pad)
    ws = torch.zeros(pa.PA_STATUS_BYTES, dtype=torch.uint8, device="cuda")
    width = heads * (576 if op == "absorb" else 128)
    outs = [outputs(rows, width, pad) for _ in range(2 if op == "expand" else 1)]
    torch.cuda.synchronize()
    first = wd.view(-1)[128 * 512:] if op == "project" else wd
    if op == "expand":
        pa.pa_mla_expand(rows, heads, xd, xd.stride(0), wd, wd.stride(0), outs[0], outs[1], outs[0].stride(0), ws, stream)
    else:
        f = pa.pa_mla_absorb if op == "absorb" else pa.pa_mla_project
        f(rows, heads, xd, xd.stride(0), first, wd.stride(0), outs[0], outs[0].stride(0), ws, stream)
    st, det = pa.pa_check(None, ws, stream)
    return x, w, outs, st, det, width


def check(op, rows, heads, **kw):
    x, w, outs, st, det, width = run(op, rows, heads, **kw)
    assert st == 0, (st, det)
    f = {"absorb": mla.absorb, "project": mla.project, "expand": mla.expand}[op]
    refs = f(f64(x), f64(w))
    mags = f(np.abs(f64(x)), np.abs(f64(w)))
    K = 128 if op == "absorb" else 512
    for out, ref, mag in zip(outs, refs if op == "expand" else [refs], mags if op == "expand" else [mags]):
        got = out[:rows, :width].double().cpu().numpy().reshape(ref.shape)
        err = np.abs(got - ref)
        tol = 2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag
        assert np.isfinite(got).all() and (err <= tol).all(), float((err / np.maximum(tol, 1e-30)).max())
        if op == "absorb":
            assert (got[..., 512:] == ref[..., 512:]).all()
        assert (out[:rows, width:] == 7).all() and (out[rows:] == 7).all()


@pytest.mark.parametrize("op", ["absorb", "project", "expand"])
@pytest.mark.parametrize("rows", ROWS)
def test_rows(op, rows):
    check(op, rows, 3, pad=8)


@pytest.mark.parametrize("op", ["absorb", "project", "expand"])
@pytest.mark.parametrize("heads", [1, 2, 5, 16, 128])
def test_heads(op, heads):
    check(op, 70, heads, w_pad=64)


@pytest.mark.parametrize("op", ["absorb", "project", "expand"])
def test_many_rows(op):
    check(op, 1500, 5, pad=64)


# sizes whose tiles CTA pairs take: blocks of 256 rows, whole and ragged, times heads
PAIRS = [(257, 192), (300, 200), (769, 96), (1025, 77), (5000, 20), (12300, 8), (33000, 3)]


@pytest.mark.parametrize("rows, heads", PAIRS)
def test_expand_by_pairs(rows, heads):
    check("expand", rows, heads, pad=8)


def test_expand_by_pairs_with_weights_apart():
    check("expand", 600, 130, w_pad=64, pad=64)


@pytest.mark.parametrize("op, rows, heads", [("absorb", 140, 2), ("project", 140, 2), ("expand", 140, 2), ("expand", 300, 192)])
def test_a_rows_nan_stays_its_own(op, rows, heads):
    shape = {"absorb": (rows, heads, 192), "project": (rows, heads, 512), "expand": (rows, 512)}[op]
    x = randn(5, *shape)
    w = randn(6, heads, 256, 512, scale=0.05)
    clean = run(op, rows, heads, x=x, w=w)[2]
    dirty = x.clone()
    dirty[7] = float("nan")
    dirty[133] = float("inf")
    got = run(op, rows, heads, x=dirty, w=w)[2]
    others = [r for r in range(rows) if r not in (7, 133)]
    for a, b in zip(clean, got):
        assert torch.equal(a[others], b[others]) and b[7].isnan().any()


@pytest.mark.parametrize("op, heads", [("absorb", 4), ("project", 4), ("expand", 4), ("expand", 200)])
def test_the_same_call_gives_the_same_bits_on_any_stream(op, heads):
    a = run(op, 300, heads)[2]
    b = run(op, 300, heads, stream=torch.cuda.Stream())[2]
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("op, rows, heads", [("absorb", 40, 2), ("project", 40, 2), ("expand", 40, 2), ("expand", 300, 192)])
def test_a_missing_load_is_reported_and_the_next_call_works(op, rows, heads):
    import paged_quantized_kv_gqa_gb300 as pa
    pa.pa_debug_set_faults(wait_limit_ns=2_000_000, skip_first_load=True)
    try:
        assert run(op, rows, heads)[3] == pa.PA_ERR_DEVICE_TIMEOUT
    finally:
        pa.pa_debug_set_faults()
    check(op, rows, heads)


@pytest.mark.parametrize("op, rows, heads", [("absorb", 50, 2), ("project", 50, 2), ("expand", 50, 2), ("expand", 300, 192)])
def test_captured(op, rows, heads):
    import paged_quantized_kv_gqa_gb300 as pa
    w = randn(8, heads, 256, 512, scale=0.05).cuda()
    shape = {"absorb": (rows, heads * 192), "project": (rows, heads * 512), "expand": (rows, 512)}[op]
    x = randn(9, *shape).cuda()
    ws = torch.zeros(pa.PA_STATUS_BYTES, dtype=torch.uint8, device="cuda")
    width = heads * (576 if op == "absorb" else 128)
    out = [torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def call():
        if op == "expand":
            pa.pa_mla_expand(rows, heads, x, 512, w, 256 * 512, out[0], out[1], width, ws)
        elif op == "absorb":
            pa.pa_mla_absorb(rows, heads, x, x.stride(0), w, 256 * 512, out[0], width, ws)
        else:
            pa.pa_mla_project(rows, heads, x, x.stride(0), w[:, 128:], 256 * 512, out[0], width, ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    x.copy_(randn(10, *shape).cuda())
    g.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in out]
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, out)) and got[0].abs().sum() > 0
