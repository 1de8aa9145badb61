"""Lists of tensors that are kept from call to call."""

import pytest
import torch

from train_ref import BF16, DEV, F32, rnd, within

pytestmark = pytest.mark.gpu


def test_a_kept_list_follows_its_tensors(lib):
    ts = [rnd(5000, seed=i, dtype=torch.float32) for i in range(3)]
    outs = [torch.zeros_like(t) for t in ts]
    kept, out = lib.tensor_list(ts), lib.tensor_list(outs)
    lib.clip_grad_norm(kept, 1.0, out=out)
    for k in range(2):
        ts[k].data = rnd(4000 - k, seed=10 + k, dtype=torch.float32)
        outs[k].data = torch.zeros_like(ts[k])
        torch.cuda.empty_cache()
        want = sum(float(t.double().square().sum()) for t in ts) ** 0.5
        assert abs(float(lib.grad_norm(kept)) - want) <= 256 * F32 * want
        lib.clip_grad_norm(kept, 1.0, out=out)
        for t, o in zip(ts, outs):
            ref = t.double() / (want + 1e-6)
            within(o, ref, 300 * F32 * ref.abs())
    g = rnd(4, 30)
    kept = lib.tensor_list([g])
    lib.clip_examples(kept, 1.0)
    g.data = rnd(3, 50, seed=4)
    (s,), sq = lib.clip_examples(kept, 1.0)
    (t,), tq = lib.clip_examples([g], 1.0)
    assert torch.equal(s, t) and torch.equal(sq, tq) and s.shape == (50,)
    assert lib.poll_status() == 0
