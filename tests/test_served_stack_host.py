"""ServedStack's checks of its arguments, before any device work: what a kernel would read or
write past a buffer for is refused."""
import pytest

torch = pytest.importorskip("torch")

D = 64


def layer(K=64, F=96, heads=2, **other):
    z = lambda n, k: (torch.zeros((n, k), dtype=torch.int8), 1.0)  # noqa: E731
    lw = {"q": z(heads * D, K), "k": z(D, K), "v": z(D, K), "o": z(K, heads * D), "gate": z(F, K), "up": z(F, K),
          "down": z(K, F), "attn_gain": torch.ones(K), "mlp_gain": torch.ones(K)}
    lw.update(other)
    return lw


@pytest.mark.parametrize("weights,why", [
    ([], "needs a layer"),
    ([layer(), layer(K=128)], "do not chain"),                     # the second layer's rows are wider
    ([layer(attn_gain=torch.ones(63))], "gains"),
    ([layer(mlp_gain=torch.ones(65))], "gains"),
    ([layer(o=(torch.zeros((64, 64), dtype=torch.int8), 1.0))], "do not chain"),
    ([layer()], "CUDA"),                                           # sound: gets as far as the device
])
def test_weights_that_do_not_fit(weights, why):
    import bit_plane_select_gb300 as t
    from bit_plane_select_gb300.stack import ServedStack
    with pytest.raises(ValueError, match=why):
        ServedStack(weights, D, t.Rope(), 4, 16, device="cpu")


@pytest.mark.parametrize("shape", [(7, 64), (6, 63), (6, 65), (1, 6, 64), (64,)])
def test_rows_that_are_not_the_plan_s(shape):
    from bit_plane_select_gb300.stack import ServedStack
    stack = ServedStack.__new__(ServedStack)
    stack.layers = [{}]
    with pytest.raises(ValueError, match="of the plan's batch"):
        stack.step([{"o": torch.empty(6, 64)}], torch.zeros(shape))
    with pytest.raises(ValueError, match="of the plan's batch"):
        stack.step([], torch.zeros(6, 64))
