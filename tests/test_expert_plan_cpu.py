"""expert_mlp refuses plans whose experts do not begin at multiples of 128 rows, also where the row
count is that of a plan that does (no GPU: the sort is done here)."""
import copy
import pickle

import pytest

torch = pytest.importorskip("torch")

import scaled_fp8_linear_amd as m  # noqa: E402

BF, i32 = torch.bfloat16, torch.int32


def sort(expert_idx, experts, multiple):
    """What fp8_moe_sort gives, with the rows that fp8_moe_rows names."""
    tokens, topk = expert_idx.shape
    flat = expert_idx.reshape(-1)
    slot = torch.full((flat.numel(),), -1, dtype=i32)
    source = torch.full((m.fp8_moe_rows(tokens, topk, experts, multiple),), -1, dtype=i32)
    counts = torch.zeros(experts, dtype=i32)
    offsets, at = torch.zeros(experts + 1, dtype=i32), 0
    for e in range(experts):
        offsets[e] = at
        for p in (flat == e).nonzero().flatten().tolist():
            row = at + int(counts[e])
            slot[p], source[row] = row, p
            counts[e] += 1
        at += -(-int(counts[e]) // multiple) * multiple
    offsets[experts] = at
    return slot.view(tokens, topk), source, counts, offsets


@pytest.fixture
def called(monkeypatch):
    """expert_plan by the sort above, and whether expert_mlp came as far as the products."""
    calls = []
    monkeypatch.setattr(m.experts._abi, "fp8_moe_sort", sort)
    monkeypatch.setattr(m.experts._ExpertMlpFn, "apply", lambda *a: calls.append(a))
    return calls


def mlp(plan, experts, up=True, down=True):
    xs = torch.zeros(plan.source.numel(), 128, dtype=BF)
    return m.expert_mlp(xs, torch.zeros(experts, 256, 128, dtype=BF, requires_grad=up),
                        torch.zeros(experts, 128, 128, dtype=BF, requires_grad=down), plan)


# an expert's pairs and a multiple whose row count is a multiple of 128 and not below that of
# multiple 128
MIXED = [([150, 50], 96), ([150, 240], 192), ([100, 100, 100], 192), ([300, 200, 100], 192)]


@pytest.mark.parametrize("per_expert,multiple", MIXED)
def test_row_counts_do_not_tell(called, per_expert, multiple):
    idx = torch.repeat_interleave(torch.arange(len(per_expert)), torch.tensor(per_expert)).view(-1, 1)
    plan = m.expert_plan(idx, len(per_expert), multiple)
    rows = plan.source.numel()
    assert rows % 128 == 0 and rows >= m.fp8_moe_rows(len(idx), 1, len(per_expert), 128)
    assert (plan.offsets % 128).any()
    bare = m.ExpertPlan(*plan)                   # nobody says what it was padded to
    for p in (plan, copy.copy(plan), pickle.loads(pickle.dumps(plan)), bare):
        with pytest.raises(ValueError, match="mix experts"):
            mlp(p, len(per_expert))
    for up, down in ((True, False), (False, True)):
        with pytest.raises(ValueError, match="mix experts"):
            mlp(bare, len(per_expert), up, down)
    assert not called
    # the products alone take any offsets, and nothing is read back
    mlp(bare, len(per_expert), False, False)
    with torch.no_grad():
        mlp(bare, len(per_expert))
        with pytest.raises(ValueError, match="mix experts"):
            mlp(plan, len(per_expert))
    assert len(called) == 2


@pytest.mark.parametrize("multiple", [128, 256, 384])
def test_whole_blocks_pass(called, multiple):
    idx = torch.tensor([0] * 150 + [1] * 50).view(100, 2)
    plan = m.expert_plan(idx, 2, multiple)
    for n, p in enumerate((plan, m.ExpertPlan(*plan), copy.copy(plan))):
        mlp(p, 2)
        assert len(called) == n + 1


def test_the_plan_stays_four_tensors(called):
    plan = m.expert_plan(torch.zeros(3, 2, dtype=torch.int64), 2, 128)
    slot, source, counts, offsets = plan
    assert len(plan) == 4 and plan.multiple == 128 and plan[3] is offsets is plan.offsets
    assert plan.slot is slot and plan.source is source and plan.counts is counts
    assert m.ExpertPlan(*plan).multiple is None
    # new offsets may be any: what the plan was made with no longer says anything
    assert plan._replace(offsets=offsets + 1).multiple is None
    with pytest.raises(ValueError, match="mix experts"):
        mlp(plan._replace(offsets=offsets + 1), 2)
