"""What the products around latent attention refuse, before any GPU work (CPU)."""
import pytest

A = 1 << 20


@pytest.fixture(scope="module")
def pa():
    import paged_quantized_kv_gqa_gb300 as m
    return m


def args(op, **kw):
    width = {"absorb": (192, 576), "project": (512, 128), "expand": (None, 128)}[op]
    a = dict(rows=5, heads=3, x=A, x_stride=512 if op == "expand" else 3 * width[0], w=A,
             w_head_stride=(256 if op == "expand" else 128) * 512, out=2 * A, out2=3 * A, out_stride=3 * width[1],
             workspace=4 * A)
    a.update(kw)
    return a


def call(pa, op, **kw):
    a = args(op, **kw)
    front = (a["rows"], a["heads"], a["x"], a["x_stride"], a["w"], a["w_head_stride"], a["out"])
    back = (a["out_stride"], a["workspace"], 0)
    {"absorb": pa.pa_mla_absorb, "project": pa.pa_mla_project, "expand": pa.pa_mla_expand}[op](
        *front, *((a["out2"],) if op == "expand" else ()), *back)


@pytest.mark.parametrize("op", ["absorb", "project", "expand"])
@pytest.mark.parametrize("kw, text", [
    (dict(rows=-1), "rows"),
    (dict(heads=0), "heads"),
    (dict(x=None), "null"),
    (dict(w=None), "null"),
    (dict(out=None), "null"),
    (dict(workspace=None), "workspace"),
    (dict(x_stride=504), "stride"),
    (dict(out_stride=376), "stride"),
    (dict(w_head_stride=128 * 512 - 8), "w_head_stride"),
    (dict(x=A + 8), "aligned"),
    (dict(w=A + 2), "aligned"),
    (dict(out=A + 4), "aligned"),
    (dict(x_stride=4097), "aligned"),
    (dict(w_head_stride=256 * 512 + 4), "aligned"),
    (dict(out_stride=4100), "aligned"),
    (dict(x_stride=1 << 40), "2\\^40"),
])
def test_refusals(pa, op, kw, text):
    with pytest.raises(pa.PaError, match=text) as e:
        call(pa, op, **kw)
    assert e.value.status == pa.PA_ERR_INVALID_ARG


def test_expand_wants_both_outputs_and_whole_heads(pa):
    for kw in (dict(out2=None), dict(out2=A + 8), dict(w_head_stride=128 * 512)):
        with pytest.raises(pa.PaError):
            call(pa, "expand", **kw)


@pytest.mark.parametrize("op", ["absorb", "project", "expand"])
def test_no_rows_is_no_work(pa, op):
    call(pa, op, rows=0, x=None, out=None, out2=None)


@pytest.mark.parametrize("op", ["absorb", "project", "expand"])
@pytest.mark.parametrize("kw", [dict(rows=1 << 32), dict(heads=(1 << 31) + 1)])
def test_sizes_beyond_the_argument(pa, op, kw):
    with pytest.raises(OverflowError):
        call(pa, op, **kw)
