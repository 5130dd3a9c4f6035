"""The layer operators' 64-bit references against their own definitions:
gradients against differences of the forward, codes against their error
bound, the transposed convolution against the forward."""
import numpy as np
import pytest

from tests import layer_reference as ref


def difference(f, x, direction, h=1e-5):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("gate", [None, "group", "channel"])
@pytest.mark.parametrize("groups", [1, 3])
def test_norm_gradients_against_differences(groups, gate):
    rng = np.random.default_rng(groups)
    rows, c, eps, alpha = 5, 24, 1e-3, 0.9
    v = dict(r=rng.normal(size=(rows, c)), y=rng.normal(size=(rows, c)), w=rng.normal(size=c),
             s=rng.normal(size=c), wn=rng.normal(size=c))
    width = {None: 0, "group": groups, "channel": c}[gate]
    v["z"] = rng.normal(size=(rows, width)) if width else None
    d_out, d_next = rng.normal(size=(rows, c)), rng.normal(size=(rows, c))

    def forward(**k):
        a = {**v, **k}
        out, u, _ = ref.norm_out(a["r"], a["y"], a["z"], a["w"], a["s"], groups, eps, alpha)
        nxt, s = ref.norm_next(out, a["wn"], groups, eps)
        return out, nxt, u, s

    out, nxt, u, s = forward()
    grads, _ = ref.norm_grads(d_out, d_next, out, s, v["y"], u, v["z"], v["w"], v["s"], v["wn"],
                              groups, alpha)
    names = dict(r="residual", y="y", w="w_post", s="scale", wn="w_next", z="gate")
    for k, name in names.items():
        if v[k] is None:
            continue
        direction = rng.normal(size=v[k].shape)

        def loss(x):
            o, n, _, _ = forward(**{k: x})
            return (o * d_out).sum() + (n * d_next).sum()

        want = difference(loss, v[k], direction)
        # a central difference: h^2 of a third derivative, and 1e-16 / h of rounding
        assert abs((grads[name] * direction).sum() - want) < 1e-6 * (1 + abs(want)), name


@pytest.mark.parametrize("seg,halo_len,dilation", [(False, 0, 1), (True, 0, 2), (True, 7, 3),
                                                   (False, 4, 2)])
def test_conv_gradients_against_differences(seg, halo_len, dilation):
    rng = np.random.default_rng(dilation)
    b, s, c, K = 2, 13, 3, 4
    x, halo = rng.normal(size=(b, s, c)), rng.normal(size=(b, halo_len, c))
    w, g = rng.normal(size=(c, K)), rng.normal(size=(b, s, c))
    ids = (rng.random((b, halo_len + s)) < 0.3).cumsum(1) if seg else None
    grads, _ = ref.conv_grads(g, x, w, dilation, ids, halo)
    bias = rng.normal(size=c)
    for name, at in dict(x=x, halo=halo, weight=w, bias=bias).items():
        if at.size == 0:
            continue
        direction = rng.normal(size=at.shape)

        def loss(v):
            a = {**dict(x=x, halo=halo, weight=w, bias=bias), name: v}
            return (g * ref.conv_forward(a["x"], a["weight"], dilation, a["bias"], ids,
                                         a["halo"])).sum()

        want = difference(loss, at, direction)  # linear: exact but for rounding
        assert abs((grads[name] * direction).sum() - want) < 1e-8 * (1 + abs(want)), name


def test_segments_that_return_to_an_id_stay_apart():
    """A pair whose ends have the same id but a boundary between them does not count."""
    seg = np.array([5, 7, 5, 5])
    assert set(ref.conv_pairs(4, 0, 2, 2, seg)) == {(0, 0, 0), (1, 1, 0), (2, 2, 0), (3, 3, 0)}
    assert (2, 3, 1) in set(ref.conv_pairs(4, 0, 1, 2, seg))


def test_codes_error_bound():
    rng = np.random.default_rng(0)
    x = ref.bf16(rng.normal(size=(64, 300)) * np.exp(rng.normal(size=(64, 1)) * 20)).astype(
        np.float32)
    codes, scales = ref.encode(x)
    assert np.abs(codes.astype(int)).max() == 127
    back = ref.decode(codes, scales)
    m = np.repeat(np.stack([np.abs(x[:, i:i + 128]).max(1) for i in (0, 128, 256)], 1), 128,
                  axis=1)[:, :300]
    assert (np.abs(back - x) <= m / 254 * (1 + 1e-5)).all()


def test_bf16_rounding():
    assert ref.bf16(1 + 2.0 ** -8) == 1.0            # a tie goes to the even side
    assert ref.bf16(1 + 3 * 2.0 ** -8) == 1 + 2.0 ** -6
    assert np.isnan(ref.bf16(np.nan)) and ref.bf16(-np.inf) == -np.inf
