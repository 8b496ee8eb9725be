"""The training step at the edges of what its documentation allows: storage that is
replaced between steps, steps with nothing between them, sizes past a launch's limits,
dispatch that needs wide fp32 layers. Limits as in tests/train_ref.py."""
import pytest
import torch

from sparse_mixture_experts_12_b200 import binding as B
from sparse_mixture_experts_12_b200 import build as BUILD
from tests import train_ref as R
from tests.test_gpu_train import DEV, _adam_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    BUILD.build()
    yield B.load()


# ------------------------------------------------------------------------- AdamW
def test_adamw_refuses_a_parameter_whose_storage_was_replaced():
    for replace in ("data", "set_"):
        ps, gs, opt = _adam_case([100, 31], torch.float32, torch.float32, 32, False, 4)
        first, was = ps[1].detach(), ps[1].clone()   # an alias keeps the old storage
        if replace == "data":
            ps[1].data = torch.zeros_like(was)
        else:
            ps[1].set_(torch.zeros_like(was))
        with pytest.raises(ValueError, match="parameter 1"):
            opt.step(gs)
        assert opt.t == 0 and torch.equal(first, was) and (ps[1] == 0).all()
        assert all((m == 0).all() for m in opt.exp_avg)
        # a new optimizer goes on from the old one's state
        two = B.AdamW(ps, lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1,
                      state=opt.state_dict())
        two.step(gs)
        rp, _, _ = R.adamw(torch.zeros_like(was), gs[1], was * 0, was * 0, 1, 0.01, 0.8, 0.95,
                           1e-6, 0.1)
        # one step from zero is lr g / (|g| + eps), a handful of fp32 roundings
        R.check(ps[1], rp, 2.0 ** -20 * rp.abs() + 1e-12, "p")


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_state_cannot_be_pulled_from_under_it(bits):
    """The state's tensors cannot be exchanged, and what happens to them leaves the memory that
    the step writes in place."""
    ps, gs, opt = _adam_case([1000], torch.float32, torch.float32, bits, False, 5)
    qs, _, ref = _adam_case([1000], torch.float32, torch.float32, bits, False, 5)
    for name in ("exp_avg", "exp_avg_sq", "master"):
        with pytest.raises(TypeError):
            getattr(opt, name)[0] = None
    opt.step(gs)
    ref.step(gs)
    size = opt.exp_avg[0].untyped_storage().nbytes()
    opt.exp_avg[0].set_(torch.empty(0, dtype=opt.exp_avg[0].dtype, device=DEV))
    torch.cuda.empty_cache()
    other = torch.full((size,), 7, dtype=torch.uint8, device=DEV)  # would take the freed block
    opt.step(gs)
    ref.step(gs)
    assert (other == 7).all() and all(torch.equal(p, q) for p, q in zip(ps, qs))
