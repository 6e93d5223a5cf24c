"""The Muon optimizer's host side: its state through a checkpoint, its checks (no GPU)."""
import copy
import io

import pytest
import torch

from linear_cross_entropy_token_gb300 import Muon


def _with_state(dtypes, seed=0):
    """Muon over 4 x 6 parameters of these types in two groups, with momenta whose bits bf16 cannot hold."""
    g = torch.Generator().manual_seed(seed)
    ps = [torch.nn.Parameter(torch.randn(4, 6, generator=g).to(dt)) for dt in dtypes]
    opt = Muon([{"params": ps[:1], "lr": 0.1}, {"params": ps[1:]}])
    for p in ps:
        opt.state[p]["momentum"] = torch.randn(4, 6, generator=g)
    return ps, opt


TYPES = [torch.bfloat16, torch.float32, torch.bfloat16]


@pytest.mark.parametrize("through", ["dict", "file"])
def test_a_checkpoint_keeps_the_momenta_bit_for_bit(through):
    ps, opt = _with_state(TYPES)
    saved = opt.state_dict()
    if through == "file":
        file = io.BytesIO()
        torch.save(saved, file)
        file.seek(0)
        saved = torch.load(file)
    qs, new = _with_state(TYPES, seed=1)
    new.load_state_dict(saved)
    for p, q in zip(ps, qs):
        got = new.state[q]["momentum"]
        assert got.dtype == torch.float32 and torch.equal(got, opt.state[p]["momentum"])
        # updated in place from here on, and not the one that was saved
        assert got.data_ptr() != opt.state[p]["momentum"].data_ptr()
    assert new.param_groups[0]["lr"] == 0.1


def test_a_checkpoint_without_some_momenta_loads():
    ps, opt = _with_state(TYPES)
    del opt.state[ps[2]]
    qs, new = _with_state(TYPES, seed=1)
    new.load_state_dict(opt.state_dict())
    assert torch.equal(new.state[qs[0]]["momentum"], opt.state[ps[0]]["momentum"]) and qs[2] not in new.state


def test_hooks_of_a_load_see_and_change_what_is_loaded():
    ps, opt = _with_state(TYPES)
    qs, new = _with_state(TYPES, seed=1)
    seen = []

    def doubled(_, state_dict):
        state_dict = dict(state_dict)
        state_dict["state"] = {i: {"momentum": 2 * s["momentum"]} for i, s in state_dict["state"].items()}
        return state_dict

    new.register_load_state_dict_pre_hook(doubled)
    new.register_load_state_dict_post_hook(lambda o: seen.append(o.state[qs[0]]["momentum"].dtype))
    new.load_state_dict(opt.state_dict())
    assert seen == [torch.float32]
    assert torch.equal(new.state[qs[0]]["momentum"], 2 * opt.state[ps[0]]["momentum"])
    new.load_state_dict(opt.state_dict())               # and a second time, with no hook of the first left
    assert seen == [torch.float32] * 2


def test_a_momentum_that_was_saved_in_fewer_bits_comes_back_as_fp32():
    ps, opt = _with_state(TYPES)
    for p in ps:
        opt.state[p]["momentum"] = opt.state[p]["momentum"].bfloat16()
    qs, new = _with_state(TYPES, seed=1)
    new.load_state_dict(opt.state_dict())
    assert all(new.state[q]["momentum"].dtype == torch.float32 for q in qs)


def test_copies_of_the_optimizer_keep_fp32_momenta():
    ps, opt = _with_state(TYPES)
    other = copy.deepcopy(opt)
    for p, q in zip(ps, (p for g in other.param_groups for p in g["params"])):
        assert torch.equal(other.state[q]["momentum"], opt.state[p]["momentum"])


def _matrix(*shape, dtype=torch.float32):
    return torch.nn.Parameter(torch.zeros(*shape, dtype=dtype))


@pytest.mark.parametrize("group", [
    dict(params=[_matrix(4)]), dict(params=[_matrix(2, 3, 4)]), dict(params=[_matrix(4, 6, dtype=torch.float16)]),
    dict(params=_matrix(4)), dict(params=[_matrix(4, 6)], lr=-1.0), dict(params=[_matrix(4, 6)], beta=2.0),
    dict(params=[_matrix(4, 6)], eps=-1.0), dict(params=[_matrix(4, 6)], weight_decay=-0.1),
    dict(params=[_matrix(4, 6)], scale="other"), dict(params=[_matrix(4, 6)], steps=0),
    dict(params=[_matrix(4, 6)], coefficients=(1.0, 2.0)), dict(params=[_matrix(4, 6)], steps="five")])
def test_every_group_is_checked(group):
    """Whether it comes with the constructor or later; a refused group leaves the optimizer as it was."""
    opt = Muon([_matrix(4, 6)])
    with pytest.raises((ValueError, TypeError)):
        opt.add_param_group(dict(group))
    assert len(opt.param_groups) == 1 and len(opt.param_groups[0]["params"]) == 1
    with pytest.raises((ValueError, TypeError)):
        Muon([dict(params=[_matrix(4, 6)]), dict(group)])
    opt.add_param_group({"params": _matrix(6, 4, dtype=torch.bfloat16), "scale": 2.0})
    assert len(opt.param_groups) == 2 and opt.param_groups[1]["scale"] == 2.0
