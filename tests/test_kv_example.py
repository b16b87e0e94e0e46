"""The decode example: append, selection and attention together, against the
oracles of each."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import kv_oracle as ko
from oracle import qsa_oracle as orc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from top_block_selection_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("paged_decode", os.path.join(ROOT, "examples", "paged_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def host_cache(layer):
    c = {n: t.view(torch.uint8).cpu().numpy() for n, t in (("k", layer.k), ("v", layer.v))}
    return dict(c, k_scale=layer.k_scale.cpu().numpy(), v_scale=layer.v_scale.cpu().numpy(),
                table=layer.table.cpu().numpy(), lens=layer.lens.cpu().numpy(), n_new=None)


@pytest.mark.parametrize("tokens,steps,k", [(200, 3, 2), (64, 65, 4)])
def test_decode_loop(example, tokens, steps, k):
    layer, (q, ids, out) = example.decode(tokens, steps, k, Hq=8, Hkv=2, D=64, block=32)
    torch.cuda.synchronize()
    c = host_cache(layer)
    total = tokens + steps
    assert layer.tokens == total == int(c["lens"][0])
    # block keys: the mean of the stored keys
    nb = -(-total // 32)
    kb = layer.kb.cpu().numpy()
    for h in range(2):
        for i in range(nb):
            page, held = c["table"][0, i], min(32, total - i * 32)
            s = c["k_scale"][page, h]
            want = (ko.decode(c["k"][page, h, :held]).sum(0).astype(np.float32) * s / np.float32(held)).astype(np.float16)
            assert np.array_equal(kb[0, h, i], want)
    # the selection: the oracle's of the same scores, the part-filled block first
    qn = q.cpu().numpy()
    got_ids = ids.cpu().numpy()
    for h in range(2):
        s_ref, _, B, _ = orc.reference_scores(qn[0][:, h * 4:h * 4 + 4], kb[0, h, :nb], total, 32)
        assert orc.selection_report(got_ids[0, h], s_ref, B, k)["ok"]
        if total % 32:
            assert got_ids[0, h, 0, 0] == nb - 1
    # attention over it
    want, _, bound = ko.attend(c, qn.astype(np.float64), 0.125, got_ids)
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= bound + 2.0 ** -11 * (np.abs(want) + bound) + 2.0 ** -25).all()


def test_every_block_chosen_is_attention_over_the_whole(example):
    layer, (q, ids, out) = example.decode(150, 2, 5, Hq=4, Hkv=1, D=128, block=32)
    c = host_cache(layer)
    want, _, bound = ko.attend(c, q.double().cpu().numpy(), 128 ** -0.5)
    assert sorted(ids.flatten().tolist()) == [0, 1, 2, 3, 4]
    for got in (out, layer.attend(q)):
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= bound + 2.0 ** -11 * (np.abs(want) + bound) + 2.0 ** -25).all()
