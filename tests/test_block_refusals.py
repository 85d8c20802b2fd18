"""What a conditioned block's operators refuse, on the host: no kernel runs here (every refusal comes before the first
CUDA call)."""

import pytest

P = 4096  # an address that is never read


@pytest.fixture(scope="module")
def ox():
    import conv2d_implicit_gemm_gb300 as m
    return m


def _block(ox, **c):
    a = dict(x=P, ldx=64, residual=P, ldr=64, sum=P, ld_sum=64, y=P, ldy=64, post=1, post_weight=P, post_bias=P, pre=2,
             pre_weight=P, pre_bias=P, eps=1e-6, gate=P, ldg=64, gate_act=0, scale=P, lds=64, shift=P, ldh=0, groups=0, per=2,
             count=2, residual_scale=1.0, branch_scale=1.0, t=4, n=64, precision=ox.PRECISION_FP16)
    ox.oidnx_block_norm(**{**a, **c})


def _axes(ox, **c):
    a = dict(q=P, q_st=256, q_sh=64, q_out=P, qo_st=256, qo_sh=64, k=P, k_st=128, k_sh=64, k_out=P, ko_st=128, ko_sh=64,
             v=0, v_st=0, v_sh=0, v_out=0, vo_st=0, vo_sh=0, norm=1, q_weight=0, k_weight=0, eps=1e-6, cos_table=P,
             sin_table=P, table_rows=8, positions=P, positions_stride=4, axes=3, pair_axes=bytes([0, 1, 2, 2] * 8), slots=0,
             cache_rows=4, t=4, hq=4, hk=2, d=64, rot=64, interleaved=0, precision=ox.PRECISION_FP16)
    ox.oidnx_qk_norm_rope_axes(**{**a, **c})


def _cross(ox, **c):
    a = dict(q=P, q_sb=0, q_st=256, q_sh=64, k=P, k_sb=0, k_st=128, k_sh=64, v=P, v_sb=0, v_st=128, v_sh=64, o=P, o_sb=0,
             o_st=256, o_sh=64, lse=0, q_lens=0, kv_lens=0, mask=0, mask_sb=0, b=1, tq=4, kv=16, hq=4, hk=2, d=64, scale=1.0,
             precision=ox.PRECISION_FP16)
    ox.oidnx_cross_attention(**{**a, **c})


INVALID, UNSUPPORTED = 1, 3
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("change,status", [
    (dict(t=-1), INVALID), (dict(n=-1), INVALID), (dict(count=-1), INVALID), (dict(x=0), INVALID), (dict(sum=0, y=0), INVALID),
    (dict(ldx=63), INVALID), (dict(ldr=63), INVALID), (dict(ld_sum=63), INVALID), (dict(ldy=63), INVALID),
    (dict(ldg=63), INVALID), (dict(lds=-1), INVALID), (dict(ldh=1), INVALID), (dict(post=3), INVALID), (dict(pre=-1), INVALID),
    (dict(gate_act=3), INVALID), (dict(per=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=INF), INVALID), (dict(residual_scale=NAN), INVALID), (dict(branch_scale=INF), INVALID), (dict(x=P + 1), INVALID),
    (dict(post_bias=P + 1), INVALID), (dict(shift=P + 1), INVALID), (dict(groups=P + 2), INVALID), (dict(precision=0), INVALID),
    (dict(precision=4), INVALID), (dict(sum_precision=3), INVALID), (dict(sum_precision=1, sum=P + 2), INVALID),
    (dict(t=2 ** 30 + 1), UNSUPPORTED), (dict(n=2 ** 30 + 1), UNSUPPORTED),
])
def test_block_norm_refuses(ox, change, status):
    with pytest.raises(ox.OidnxError) as e:
        _block(ox, **change)
    assert e.value.status == status and "block_norm" in str(e.value)


@pytest.mark.parametrize("change,status", [
    (dict(t=-1), INVALID), (dict(hq=-1), INVALID), (dict(d=0), INVALID), (dict(rot=3), INVALID), (dict(rot=66, pair_axes=bytes(33)), INVALID),
    (dict(q=0), INVALID), (dict(q_out=0), INVALID), (dict(k_out=0), INVALID), (dict(v=P), INVALID), (dict(v_out=P), INVALID),
    (dict(cos_table=0), INVALID), (dict(positions=0), INVALID), (dict(eps=-1.0), INVALID), (dict(precision=0), INVALID),
    (dict(precision=4), INVALID), (dict(q=P + 1), INVALID), (dict(positions=P + 2), INVALID), (dict(axes=0), INVALID),
    (dict(axes=9), INVALID), (dict(axes=2), INVALID), (dict(positions_stride=3), INVALID),
    (dict(pair_axes=bytes([0] * 31 + [3])), INVALID), (dict(hq=70000), UNSUPPORTED), (dict(t=2 ** 30 + 1), UNSUPPORTED),
    (dict(d=514, rot=514, pair_axes=bytes(257)), UNSUPPORTED),
])
def test_axes_refuses(ox, change, status):
    with pytest.raises(ox.OidnxError) as e:
        _axes(ox, **change)
    assert e.value.status == status and "qk_norm_rope_axes" in str(e.value)


def test_axes_of_too_few_pairs_or_of_no_bytes(ox):
    with pytest.raises(ValueError):
        _axes(ox, pair_axes=bytes(31))
    with pytest.raises(TypeError):
        _axes(ox, pair_axes=[0] * 32)


@pytest.mark.parametrize("change,status", [
    (dict(b=-1), INVALID), (dict(tq=-1), INVALID), (dict(kv=-1), INVALID), (dict(hk=0), INVALID), (dict(hq=5), INVALID),
    (dict(d=0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(q=0), INVALID), (dict(k=0), INVALID),
    (dict(v=0), INVALID), (dict(o=0), INVALID), (dict(k=P + 1), INVALID), (dict(lse=P + 2), INVALID),
    (dict(kv_lens=P + 1), INVALID), (dict(mask=P, mask_sb=15), INVALID), (dict(precision=0), INVALID),
    (dict(precision=1), UNSUPPORTED), (dict(d=257), UNSUPPORTED), (dict(b=100000, tq=100000), UNSUPPORTED),
    (dict(kv=2 ** 30 + 1), UNSUPPORTED), (dict(tq=2 ** 29, hq=4, hk=1), UNSUPPORTED),
])
def test_cross_attention_refuses(ox, change, status):
    with pytest.raises(ox.OidnxError) as e:
        _cross(ox, **change)
    assert e.value.status == status and "cross_attention" in str(e.value)


def test_empty_calls_do_nothing(ox):
    _block(ox, t=0)
    _block(ox, n=0)
    _block(ox, count=0)
    _axes(ox, t=0)
    _axes(ox, hq=0, hk=0)
    _cross(ox, b=0)
    _cross(ox, tq=0)
    _cross(ox, hq=0)
    assert ox.oidnx_last_error() == ""


@pytest.mark.parametrize("call,count", [("oidnx_block_norm", 31), ("oidnx_qk_norm_rope_axes", 40), ("oidnx_cross_attention", 29)])
def test_calls_count_their_arguments(ox, call, count):
    with pytest.raises(TypeError):
        getattr(ox._calls, call)(*[0] * count)
