"""expert_mlp makes the copies that a backward reads (transposed codes, the 8-bit activation input) only
for the gradients that can be asked for: none without a graph. The kernels are stand-ins that tell
what they were asked for."""
import pytest

torch = pytest.importorskip("torch")

import scaled_fp8_linear_amd as m  # noqa: E402

E, COLS, HIDDEN, ROWS = 2, 128, 256, 384
BF, i32 = torch.bfloat16, torch.int32


@pytest.fixture
def asked(monkeypatch):
    asked = {}

    def quantize(x, gran, want_q_t, want_amax):
        name = {(ROWS, COLS): "x", (E * 2 * HIDDEN, COLS): "up", (E * COLS, HIDDEN): "down"}[x.shape]
        asked[name] = want_q_t
        r, c = x.shape
        t = (torch.empty(c, r, dtype=torch.uint8), torch.empty(c if name == "x" else c // 128, r // 128))
        s = torch.empty(r if name == "x" else r // 128, c // 128)
        return (torch.empty(r, c, dtype=torch.uint8), t[0] if want_q_t else None, None, s,
                t[1] if want_q_t else None)

    def act(h, act, gated, want_q_t, want_checkpoint):
        asked.update(a=want_q_t, h=want_checkpoint)
        return (None,) * 6

    monkeypatch.setattr(m.experts._abi, "fp8_quantize_amax", quantize)
    monkeypatch.setattr(m.experts._abi, "fp8_act_quantize", act)
    monkeypatch.setattr(m.experts._abi, "fp8_grouped_linear_fwd",
                        lambda q, w, *a, **k: torch.zeros(ROWS, w.shape[1], dtype=BF))
    return asked


@pytest.mark.parametrize("no_graph", [None, torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("x,up,down", [(1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0), (0, 1, 1)])
def test_copies(asked, no_graph, x, up, down):
    xs = torch.zeros(ROWS, COLS, dtype=BF, requires_grad=bool(x))
    w_up = torch.zeros(E, 2 * HIDDEN, COLS, dtype=BF, requires_grad=bool(up))
    w_down = torch.zeros(E, COLS, HIDDEN, dtype=BF, requires_grad=bool(down))
    plan = m.ExpertPlan(torch.zeros(50, 2, dtype=i32), torch.zeros(ROWS, dtype=i32),
                        torch.zeros(E, dtype=i32), torch.zeros(E + 1, dtype=i32))
    if no_graph is None:
        y = m.expert_mlp(xs, w_up, w_down, plan)
    else:
        with no_graph():
            y = m.expert_mlp(xs, w_up, w_down, plan)
        x = up = down = 0
    assert y.requires_grad == bool(x or up or down)
    # dx reads both stacks transposed and h; w_up's gradient x, h and w_down's stack; w_down's a
    assert asked == {"x": bool(up), "up": bool(x), "a": bool(down), "h": bool(x or up),
                     "down": bool(x or up)}
