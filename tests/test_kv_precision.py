"""GPU tests of what the cache attention holds in fewer bits than fp32: its
probabilities and queries (sums of 8-bit terms where there are few rows, 16-bit
ones where there are many). Errors may not grow with the context, nor with the
scales and dimensions that carry no weight.

Tolerances come from the contract (include/qsa.h): a probability times its
value scale is off by at most U of itself or F of the largest among the RUN
tokens around it, U = 2^-12, F = 2^-22, RUN = 1,024 of fp16 calls and 2^-9,
2^-19, 512 of bf16 calls."""
import numpy as np
import pytest

import kv_cases as kc
from oracle import kv_oracle as ko
from test_kv_parity import UNIT, dev, on_gpu, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = {"f16": 2.0 ** -12, "bf16": 2.0 ** -9}
F = {"f16": 2.0 ** -22, "bf16": 2.0 ** -19}
RUN = {"f16": 1024, "bf16": 512}


def one_head(B, k, v, ks, vs, block, seed=0):
    """B sequences in the same pages (one KV head) of code values k, v
    [tokens, D] and block scales ks, vs."""
    tokens, D = k.shape
    pages = -(-tokens // block)
    order = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    c = dict(table=np.broadcast_to(order, (B, pages)).copy(), lens=np.full(B, tokens, np.int32), n_new=None)
    for name, x, s in (("k", k, ks), ("v", v, vs)):
        full = np.full((pages * block, D), 0x7F, np.uint8)
        full[:tokens] = ko.encode(x)
        c[name] = np.empty((pages, 1, block, D), np.uint8)
        c[name][order, 0] = full.reshape(pages, block, D)
        c[name + "_scale"] = np.empty((pages, 1), np.float32)
        c[name + "_scale"][order, 0] = s
    return c


def rounded(x, dtype):
    return x.astype(np.float16).astype(np.float64) if dtype == "f16" else kc.as_bf16(x.astype(np.float32)).astype(np.float64)


def expected(c, q, b, j, n, scale, dtype):
    """(result, rms error of each of its elements before its rounding) of a row:
    each probability off by a uniform error of its bound, the scores' fp32 sums
    and exp2 by 2^-20 (1 + |x|) of it."""
    seen = ko.seen_tokens(c, b, j, n)
    page, off = np.array([t[0] for t in seen]), np.array([t[1] for t in seen])
    kk = ko.decode(c["k"][page, 0, off]) * c["k_scale"][page, 0].astype(np.float64)[:, None]
    code, vs = ko.decode(c["v"][page, 0, off]), c["v_scale"][page, 0].astype(np.float64)
    x = scale * (kk @ q.astype(np.float64))
    p = np.exp(x - x.max())
    w = p * vs
    d = np.maximum(U[dtype] * w, F[dtype] * w.max()) + 2.0 ** -20 * (1 + np.abs(x - x.max())) * w
    return (w @ code) / p.sum(), np.sqrt((d * d / 3) @ (code * code)) / p.sum()


def check_norm(tbs, c, q, dtype, rows, scale, kernel):  # noqa: F811
    """The error's norm over these rows is that of the bounds' uniform errors and
    of the result's rounding, give or take a quarter."""
    args, _ = on_gpu(c)
    got = tbs.qsa_kv_attend(dev(q, dtype), *args, scale=scale)
    assert kernel + " " in tbs.qsa_arm() + " "
    got = got.double().cpu().numpy()
    err = room = 0.0
    for b, j, h in rows:
        want, rms = expected(c, q[b, j, h], b, j, q.shape[1], scale, dtype)
        err += ((got[b, j, h] - want) ** 2).sum()
        room += (rms ** 2).sum() + ((rounded(want, dtype) - want) ** 2).sum()
    assert np.sqrt(err) <= 1.25 * np.sqrt(room), (np.sqrt(err), np.sqrt(room))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_errors_do_not_grow_with_the_context(tbs, dtype):  # noqa: F811
    """49,152 tokens for each CTA, scores of standard deviation 0.4 to 3 by block."""
    rng = np.random.default_rng(1)
    tokens, D, block = 49152, 64, 128
    pages = tokens // block
    ks, vs = 2.0 ** rng.integers(-8, -4, pages), 2.0 ** rng.integers(-8, -5, pages)
    c = one_head(152, rng.standard_normal((tokens, D)) * 100, rng.standard_normal((tokens, D)) * 100, ks, vs, block)
    q = kc.ROUND[dtype](rng.standard_normal((152, 1, 4, D)))
    rows = [(int(b), 0, int(h)) for b, h in zip(rng.integers(152, size=24), rng.integers(4, size=24))]
    check_norm(tbs, c, q, dtype, rows, D ** -0.5, "kv_attend_kernel")


@pytest.mark.parametrize("n,R", [(1, 4), (1, 16), (1, 32), (64, 2)])
@pytest.mark.parametrize("dtype,bits", [("f16", 18.2), ("f16", 22.5), ("bf16", 15.2), ("bf16", 19.5)])
def test_one_token_above_very_many(tbs, dtype, bits, n, R):  # noqa: F811
    """One token whose score is `bits` (in log2) above those of 49,151 equal ones,
    which together still carry some weight: value -1 against 1."""
    tokens, D, block = 49152, 64, 128
    k, v = np.zeros((tokens, D)), np.ones((tokens, D))
    k[5, 0], v[5] = 1.0, -1.0
    c = one_head(152, k, v, np.ones(tokens // block), np.ones(tokens // block), block)
    q = np.zeros((152, n, R, D))
    q[..., 0] = 1.0
    scale = bits * np.log(2.0)
    args, _ = on_gpu(c)
    got = tbs.qsa_kv_attend(dev(q, dtype), *args, scale=scale).double().cpu().numpy()
    rest = (tokens - n + np.arange(n)) * 2.0 ** -bits  # the weight of the others, for each row
    want = ((rest - 1) / (rest + 1))[None, :, None, None]
    tol = U[dtype] + RUN[dtype] * F[dtype] + UNIT[dtype] + 2.0 ** -16
    assert np.abs(got - want).max() <= tol, (float(np.abs(got - want).max()), tol)


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,n,R,far", [(128, 1, 4, 14), (64, 1, 32, 14), (128, 128, 16, 26), (64, 128, 16, 26)])
def test_large_value_scale_without_weight(tbs, D, dtype, n, R, far, at):  # noqa: F811
    """A block whose values are 2^far times the others' and whose scores lie 60
    (in log2) below them changes nothing, whether a row sees it or not."""
    rng = np.random.default_rng(D + n)
    tokens, block = 2000, 64
    pages = -(-tokens // block)
    k, v = rng.standard_normal((tokens, D)), rng.standard_normal((tokens, D)) * 100
    i = {"first": 0, "middle": pages // 2, "last": pages - 1}[at]
    k[:, 0] = 0.0
    k[i * block:(i + 1) * block, 0] = -15.0
    vs = np.full(pages, 2.0 ** -12)
    vs[i] = 2.0 ** (far - 12)
    c = one_head(1, k, v, np.ones(pages), vs, block)
    q = rng.standard_normal((1, n, R, D)) * D ** -0.5
    q[..., 0] = 60 * np.log(2.0) / 15
    q = kc.ROUND[dtype](q)
    rows = [(0, int(j), int(h)) for j, h in zip(rng.integers(n, size=40), rng.integers(R, size=40))]
    check_norm(tbs, c, q, dtype, rows, 1.0, "kv_attend_kernel" if n == 1 else "kv_attend_many_kernel")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,n,R", [(64, 1, 4), (128, 1, 16), (128, 64, 32)])
def test_query_dimension_far_above_the_others(tbs, dtype, D, n, R):  # noqa: F811
    """One dimension of the queries 512 times the others, where the keys are
    zero: the scores are those of the other dimensions."""
    rng = np.random.default_rng(n)
    tokens, block = 1500, 64
    pages = -(-tokens // block)
    k, v = rng.standard_normal((tokens, D)) * 4, rng.standard_normal((tokens, D)) * 100
    k[:, 3] = 0.0
    c = one_head(1, k, v, np.full(pages, 0.25), np.full(pages, 2.0 ** -6), block)
    q = rng.standard_normal((1, n, R, D)) * 4
    q[..., 3] = 512 * 4
    q = kc.ROUND[dtype](q)
    rows = [(0, int(j), int(h)) for j, h in zip(rng.integers(n, size=40), rng.integers(R, size=40))]
    check_norm(tbs, c, q, dtype, rows, D ** -0.5, "kv_attend_kernel" if n == 1 else "kv_attend_many_kernel")


@pytest.mark.parametrize("kind", ["zeros first", "zeros far above 30", "zeros far above 45", "rising", "falling"])
@pytest.mark.parametrize("D,n,R", [(128, 1, 4), (64, 1, 32), (128, 128, 16), (64, 128, 16)])
def test_weights_far_apart(tbs, D, n, R, kind):  # noqa: F811
    """Blocks of zeros (the smallest scale there is) before all others, or 30
    and 45 (in log2) above all others in the score; value scales that rise or
    fall by 2^3 from block to block."""
    rng = np.random.default_rng(D + n)
    tokens, block = 2000, 64
    pages = -(-tokens // block)
    k, v = rng.standard_normal((tokens, D)), rng.standard_normal((tokens, D)) * 100
    k[:, 0] = 0.0
    vs = np.full(pages, 2.0 ** -6)
    if kind.startswith("zeros"):
        i = 0 if kind == "zeros first" else 3
        v[i * block:(i + 1) * block] = 0.0
        vs[i] = 2.0 ** -100
        if i:
            k[i * block:(i + 1) * block, 0] = 15.0
    else:
        vs = 2.0 ** (3.0 * np.arange(pages) - 40)[::1 if kind == "rising" else -1]
    c = one_head(1, k, v, np.ones(pages), vs, block)
    q = rng.standard_normal((1, n, R, D)) * D ** -0.5
    q[..., 0] = (45 if kind.endswith("45") else 30) * np.log(2.0) / 15
    q = kc.ROUND["bf16"](q)
    rows = [(0, int(j), int(h)) for j, h in zip(rng.integers(n, size=40), rng.integers(R, size=40))]
    check_norm(tbs, c, q, "bf16", rows, 1.0, "kv_attend_kernel" if n == 1 else "kv_attend_many_kernel")
