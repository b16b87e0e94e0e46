"""GPU tests of what the 4-bit cache's attention holds in fewer bits than fp32,
as tests/test_kv_precision.py has them of the 8-bit cache, with a scale for
each token. Tolerances come from the contract (include/qsa.h): a probability
times its value scale is off by at most U of itself or F of the largest among
the RUN tokens around it, U = 2^-12, F = 2^-22, RUN = 1,024 of fp16 calls and
2^-9, 2^-19, 512 of bf16 calls; RUN is twice that of 64 dimensions."""
import numpy as np
import pytest

import kv4_cases as kc
from oracle import kv4_oracle as ko
from test_kv4_parity import UNIT, dev, on_gpu, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = {"f16": 2.0 ** -12, "bf16": 2.0 ** -9}
F = {"f16": 2.0 ** -22, "bf16": 2.0 ** -19}
RUN = {"f16": 1024, "bf16": 512}


def one_head(B, k, v, ks, vs, block, seed=0):
    """B sequences in the same pages (one KV head) of code values k, v [tokens, D] and scales ks, vs [tokens]."""
    tokens, D = k.shape
    pages = -(-tokens // block)
    order = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    c = dict(table=np.broadcast_to(order, (B, pages)).copy(), lens=np.full(B, tokens, np.int32), n_new=None)
    for name, x, s in (("k", k, ks), ("v", v, vs)):
        codes, scale = np.zeros((pages * block, D // 2), np.uint8), np.full(pages * block, np.nan, np.float32)
        codes[:tokens], scale[:tokens] = ko.encode(x), kc.as_bf16(np.asarray(s, np.float32))
        c[name], c[name + "_scale"] = np.empty((pages, 1, block, D // 2), np.uint8), np.empty((pages, 1, block), np.float32)
        c[name][order, 0], c[name + "_scale"][order, 0] = codes.reshape(pages, block, -1), scale.reshape(pages, block)
    return c


def rounded(x, dtype):
    return x.astype(np.float16).astype(np.float64) if dtype == "f16" else kc.as_bf16(x.astype(np.float32)).astype(np.float64)


def expected(c, q, b, slot, scale, dtype):
    """(result, rms error of each of its elements before its rounding) of a row:
    each probability off by a uniform error of its bound, the scores' fp32 sums
    and exp2 by 2^-20 (1 + |x|) of it."""
    slots = ko.seen_slots(c, b, slot)
    kk, ks = ko.gathered(c, b, 0, slots, "k")
    code, vs = ko.gathered(c, b, 0, slots, "v")
    x = scale * ((kk * ks[:, None]) @ q.astype(np.float64))
    p = np.exp(x - x.max())
    w = p * vs
    d = np.maximum(U[dtype] * w, F[dtype] * w.max()) + 2.0 ** -20 * (1 + np.abs(x - x.max())) * w
    return (w @ code) / p.sum(), np.sqrt((d * d / 3) @ (code * code)) / p.sum()


def check_norm(tbs, c, q, dtype, scale, kernel, seed=0):  # noqa: F811
    """The error's norm over 40 rows is that of the bounds' uniform errors and of
    the result's rounding, give or take a quarter."""
    B, n, R, _ = q.shape
    if "many" in kernel:
        kc.roomy(c, B * n * R)
    args, _ = on_gpu(c)
    got = tbs.qsa_kv4_attend(dev(q, dtype), *args, scale=scale)
    assert kernel + " " in tbs.qsa_arm() + " "
    got = got.double().cpu().numpy()
    rng, err, room = np.random.default_rng(seed), 0.0, 0.0
    for _ in range(40):
        b, j, h = int(rng.integers(B)), int(rng.integers(n)), int(rng.integers(R))
        want, rms = expected(c, q[b, j, h], b, int(c["lens"][b]) - n + j, scale, dtype)
        err += ((got[b, j, h] - want) ** 2).sum()
        room += (rms ** 2).sum() + ((rounded(want, dtype) - want) ** 2).sum()
    assert np.sqrt(err) <= 1.25 * np.sqrt(room), (np.sqrt(err), np.sqrt(room))


FORMS = [(128, 1, 4, "kv4_attend_kernel"), (64, 1, 16, "kv4_attend_kernel"), (128, 128, 16, "kv4_attend_many_kernel"),
         (64, 128, 16, "kv4_attend_many_kernel")]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_errors_do_not_grow_with_the_context(tbs, dtype, D):  # noqa: F811
    """49,152 tokens for each CTA, scores of standard deviation about 1, scales spread by token."""
    rng = np.random.default_rng(1)
    tokens = 49152
    c = one_head(152, rng.standard_normal((tokens, D)) * 2, rng.standard_normal((tokens, D)) * 2,
                 0.5 * 2.0 ** rng.uniform(-2, 1, tokens), 2.0 ** rng.uniform(-3, 1, tokens), 128)
    q = kc.ROUND[dtype](rng.standard_normal((152, 1, 4, D)))
    check_norm(tbs, c, q, dtype, D ** -0.5, "kv4_attend_kernel")


@pytest.mark.parametrize("D,n,R", [(64, 1, 4), (128, 1, 16), (64, 1, 16), (128, 64, 2)])
@pytest.mark.parametrize("dtype,bits", [("f16", 18.2), ("f16", 22.5), ("bf16", 15.2), ("bf16", 19.5)])
def test_one_token_above_very_many(tbs, dtype, bits, D, n, R):  # noqa: F811
    """One token whose score is `bits` (in log2) above those of 49,151 equal ones,
    which together still carry some weight: value -1 against 1."""
    tokens = 49152
    k, v = np.zeros((tokens, D)), np.ones((tokens, D))
    k[5, 0], v[5] = 1.0, -1.0
    c = one_head(152, k, v, np.ones(tokens), np.ones(tokens), 128)
    q = np.zeros((152, n, R, D))
    q[..., 0] = 1.0
    args, _ = on_gpu(c)
    got = tbs.qsa_kv4_attend(dev(q, dtype), *args, scale=bits * np.log(2.0)).double().cpu().numpy()
    rest = (tokens - n + np.arange(n)) * 2.0 ** -bits  # the weight of the others, for each row
    want = ((rest - 1) / (rest + 1))[None, :, None, None]
    tol = U[dtype] + RUN[dtype] * (128 // D) * F[dtype] + UNIT[dtype] + 2.0 ** -16
    assert np.abs(got - want).max() <= tol, (float(np.abs(got - want).max()), tol)


@pytest.mark.parametrize("at", [0, 1000, 1999])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,n,R,kernel", FORMS)
def test_large_value_scale_without_weight(tbs, D, dtype, n, R, kernel, at):  # noqa: F811
    """A token whose values are 2^14 (of many rows 2^26) times the others' and whose
    score lies 60 (in log2) below them changes nothing, whether a row sees it or not."""
    rng = np.random.default_rng(D + n)
    k, v = rng.standard_normal((2000, D)), rng.standard_normal((2000, D)) * 2
    k[:, 0] = 0.0
    k[at, 0] = -6.0
    vs = 2.0 ** rng.uniform(-8, -7, 2000)
    vs[at] = 2.0 ** ((14 if n == 1 else 26) - 8)
    c = one_head(1, k, v, np.ones(2000), vs, 64)
    q = rng.standard_normal((1, n, R, D)) * D ** -0.5
    q[..., 0] = 60 * np.log(2.0) / 6
    check_norm(tbs, c, kc.ROUND[dtype](q), dtype, 1.0, kernel)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,n,R,kernel", FORMS)
def test_query_dimension_far_above_the_others(tbs, dtype, D, n, R, kernel):  # noqa: F811
    """One dimension of the queries 512 times the others, where the keys are zero."""
    rng = np.random.default_rng(n)
    k, v = rng.standard_normal((1500, D)) * 2, rng.standard_normal((1500, D)) * 2
    k[:, 3] = 0.0
    c = one_head(1, k, v, np.full(1500, 0.5), 2.0 ** rng.uniform(-6, -5, 1500), 64)
    q = rng.standard_normal((1, n, R, D)) * 4
    q[..., 3] = 512 * 4
    check_norm(tbs, c, kc.ROUND[dtype](q), dtype, D ** -0.5, kernel)


@pytest.mark.parametrize("kind", ["zeros first", "zeros far above 30", "zeros far above 45", "rising", "falling"])
@pytest.mark.parametrize("D,n,R,kernel", FORMS)
def test_weights_far_apart(tbs, D, n, R, kernel, kind):  # noqa: F811
    """Tokens of zeros (the smallest scale there is) before all others, or 30 and 45
    (in log2) above all others in the score; value scales that rise or fall by 2^3
    every 64 tokens."""
    rng = np.random.default_rng(D + n)
    tokens = 2000
    k, v = rng.standard_normal((tokens, D)), rng.standard_normal((tokens, D)) * 2
    k[:, 0] = 0.0
    vs = np.full(tokens, 2.0 ** -6)
    if kind.startswith("zeros"):
        at = slice(0, 64) if kind == "zeros first" else slice(192, 256)
        v[at] = 0.0
        vs[at] = 2.0 ** -100
        if kind != "zeros first":
            k[at, 0] = 6.0
    else:
        vs = 2.0 ** (3.0 * (np.arange(tokens) // 64) - 40)[::1 if kind == "rising" else -1]
    c = one_head(1, k, v, np.ones(tokens), vs, 64)
    q = rng.standard_normal((1, n, R, D)) * D ** -0.5
    q[..., 0] = (45 if kind.endswith("45") else 30) * np.log(2.0) / 6
    check_norm(tbs, c, kc.ROUND["bf16"](q), "bf16", 1.0, kernel)
