"""What the token operators refuse, on the host: no kernel runs here (every refusal comes before the first CUDA call)."""

import pytest

P = 4096  # an address that is never read


@pytest.fixture(scope="module")
def ox():
    import conv2d_implicit_gemm_gb300 as m
    return m


def _linear(ox, **c):
    a = dict(x=P, ldx=64, w=P, ldw=64, bias=0, residual=0, ldr=0, y=P, ldy=32, m=4, n=32, k=64, act=0,
             precision=ox.PRECISION_FP16)
    ox.oidnx_linear(**{**a, **c})


def _norm(ox, **c):
    a = dict(q=P, q_st=256, q_sh=64, q_out=P, qo_st=256, qo_sh=64, k=P, k_st=128, k_sh=64, k_out=P, ko_st=128, ko_sh=64,
             v=0, v_st=0, v_sh=0, v_out=0, vo_st=0, vo_sh=0, q_weight=0, k_weight=0, eps=1e-6, cos_table=P, sin_table=P,
             table_rows=8, positions=P, slots=0, cache_rows=4, t=4, hq=4, hk=2, d=64, rot=64, interleaved=0,
             precision=ox.PRECISION_FP16)
    ox.oidnx_qk_norm_rope(**{**a, **c})


def _attn(ox, **c):
    a = dict(q=P, q_sb=0, q_st=256, q_sh=64, k=P, k_sb=0, k_st=128, k_sh=64, v=P, v_sb=0, v_st=128, v_sh=64, o=P, o_sb=0,
             o_st=256, o_sh=64, lse=0, q_lens=0, kv_lens=0, b=1, tq=4, cap=16, hq=4, hk=2, d=64, window=0, sinks=0,
             scale=1.0, precision=ox.PRECISION_FP16)
    ox.oidnx_window_attention(**{**a, **c})


INVALID, UNSUPPORTED = 1, 3


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(k=-2), INVALID), (dict(x=0), INVALID), (dict(w=0), INVALID),
    (dict(y=0), INVALID), (dict(ldx=63), INVALID), (dict(ldw=63), INVALID), (dict(ldy=31), INVALID),
    (dict(residual=P, ldr=31), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(x=P + 1), INVALID),
    (dict(bias=P + 1), INVALID), (dict(y=P + 1), INVALID), (dict(precision=0), INVALID), (dict(precision=4), INVALID),
    (dict(precision=1), UNSUPPORTED), (dict(m=2 ** 30 + 1), UNSUPPORTED), (dict(n=2 ** 30 + 1, ldy=2 ** 31), UNSUPPORTED),
])
def test_linear_refuses(ox, change, status):
    with pytest.raises(ox.OidnxError) as e:
        _linear(ox, **change)
    assert e.value.status == status and "linear" in str(e.value)


@pytest.mark.parametrize("change,status", [
    (dict(t=-1), INVALID), (dict(hq=-1), INVALID), (dict(d=0), INVALID), (dict(rot=3), INVALID), (dict(rot=66), INVALID),
    (dict(q=0), INVALID), (dict(q_out=0), INVALID), (dict(k_out=0), INVALID), (dict(v=P), INVALID),
    (dict(v_out=P), INVALID), (dict(cos_table=0), INVALID), (dict(positions=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(precision=0), INVALID), (dict(precision=4), INVALID),
    (dict(q=P + 1), INVALID), (dict(positions=P + 2), INVALID), (dict(hq=70000), UNSUPPORTED),
    (dict(t=2 ** 30 + 1), UNSUPPORTED),
])
def test_norm_refuses(ox, change, status):
    with pytest.raises(ox.OidnxError) as e:
        _norm(ox, **change)
    assert e.value.status == status and "qk_norm_rope" in str(e.value)


@pytest.mark.parametrize("change,status", [
    (dict(b=-1), INVALID), (dict(tq=-1), INVALID), (dict(cap=-1), INVALID), (dict(hk=0), INVALID), (dict(hq=5), INVALID),
    (dict(d=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
    (dict(o=0), INVALID), (dict(k=P + 1), INVALID), (dict(lse=P + 2), INVALID), (dict(kv_lens=P + 1), INVALID),
    (dict(precision=0), INVALID), (dict(precision=1), UNSUPPORTED), (dict(d=257), UNSUPPORTED),
    (dict(b=100000, tq=100000), UNSUPPORTED), (dict(cap=2 ** 30 + 1), UNSUPPORTED),
])
def test_attention_refuses(ox, change, status):
    with pytest.raises(ox.OidnxError) as e:
        _attn(ox, **change)
    assert e.value.status == status and "window_attention" in str(e.value)


def test_empty_calls_do_nothing(ox):
    _linear(ox, m=0)
    _linear(ox, n=0, ldy=0)
    _norm(ox, t=0)
    _norm(ox, hq=0, hk=0)
    _attn(ox, b=0)
    _attn(ox, tq=0)
    _attn(ox, hq=0)
    assert ox.oidnx_last_error() == ""


@pytest.mark.parametrize("count", [14, 16])
def test_calls_count_their_arguments(ox, count):
    with pytest.raises(TypeError):
        ox._calls.oidnx_linear(*[0] * count)


def test_calls_refuse_what_no_c_int_holds(ox):
    with pytest.raises(OverflowError):
        _linear(ox, m=2 ** 31)
