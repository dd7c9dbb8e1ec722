"""What a ServedStack's plans hold on the device, beside the caches: layers run in turn, so a plan's layers share
what no later one reads."""
import pytest

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402
from test_gpu_attn_paged import BF, t  # noqa: E402,F401
from test_gpu_served_stack_exact import layer  # noqa: E402

pytestmark = pytest.mark.gpu
K, D, HQ, HK, PAGE = 192, 64, 4, 2, 16


def stack_of(t, layers, bits, pages):  # noqa: F811
    from bit_plane_select_gb300.stack import ServedStack
    ang = torch.arange(9000, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    return ServedStack([layer(9 + i) for i in range(layers)], D, t.Rope(ang.cos().float().cuda(), ang.sin().float().cuda()),
                       pages, PAGE, dtype=BF, cache_bits=bits)


@pytest.mark.parametrize("bits", [4, 16])
def test_one_workspace_for_a_plan_s_layers(t, bits):  # noqa: F811
    """A prefix that many rows read is written into the workspace: once, not once a layer.  Results as with a
    workspace each."""
    g = torch.Generator().manual_seed(2)
    P, B, layers = 8000, 160, 3
    pages, pre, table = ref.make_batch(g, [3] * B, 1, PAGE, P)
    stack = stack_of(t, layers, bits, pages)
    for L in stack.layers:                   # a prefix of any values
        c = L["cache"]
        for x in (c.k, c.v):
            x.copy_(torch.randint(256, x.shape, generator=g, dtype=torch.uint8) if bits == 4 else
                    torch.randn(x.shape, generator=g).to(BF))
        for x in (c.k_scale, c.v_scale) if bits == 4 else ():
            x.copy_(torch.tensor([0.1, -0.75], dtype=torch.float16).expand(x.shape))
    batch = t.KvBatch(table.cuda(), torch.full((B,), 3, dtype=torch.int32).cuda(), 1, prefix_table=pre.cuda(), prefix_len=P)
    plan = stack.plan(batch)
    assert len({p["attend"].workspace.data_ptr() for p in plan}) == 1
    if bits == 4:
        assert plan[0]["attend"].workspace.numel() > 8 * P * HK * D
    x = torch.randn(B, K, generator=g).cuda()
    got = stack.step(plan, x.clone())
    apart = stack.plan(batch)
    for L, p in zip(stack.layers, apart):
        job = (t.Attn4Job if bits == 4 else t.AttnJob)(L["cache"], batch, p["q_rot"], p["attn"])
        p["calls"][1] = (p["calls"][1][0], job)
    want = stack.step(apart, x.clone())
    torch.cuda.synchronize()
    assert torch.equal(got, want) and int(stack.err.item()) == 0 and bool(got.isfinite().all())


def test_a_prompt_plan_s_layers_share_buffers(t):  # noqa: F811
    """The products' buffers for a prompt's rows are there once for layers of one size; the first layer's results do
    not change as more layers follow."""
    g = torch.Generator().manual_seed(3)
    total = [300, 41]
    pages, _, table = ref.make_batch(g, total, 1, PAGE)
    lens = torch.tensor(total, dtype=torch.int32).cuda()
    starts = torch.tensor([0, 300, 341], dtype=torch.int32).cuda()
    x = torch.randn(341, K, generator=g).cuda()
    plans, outs = [], []
    for layers in (1, 2, 3):
        stack = stack_of(t, layers, 4, pages)
        plan = stack.prompt_plan(t.KvBatch(table.cuda(), lens, 300), 341, starts, 341, starts)
        outs.append(stack.step(plan, x.clone()))
        torch.cuda.synchronize()
        assert int(stack.err.item()) == 0
        plans.append(plan)
    for name in ("x_i8", "a_i8", "h_i8", "s", "sa", "sh", "q", "k", "v", "o", "down", "gate", "up"):
        assert len({p[name].data_ptr() for p in plans[2]}) == 1, name
    for name in ("q_rot", "attn"):
        assert len({p[name].data_ptr() for p in plans[2]}) == 3
        assert all(torch.equal(a[name], b[name]) for a, b in zip(plans[2], plans[1]))
        assert torch.equal(plans[0][0][name], plans[1][0][name])
    # the layers one by one, a plan each, on the caches of the last stack
    y = x.clone()
    every = list(stack.layers)
    for L in every:
        stack.layers = [L]
        stack.step(stack.prompt_plan(t.KvBatch(table.cuda(), lens, 300), 341, starts, 341, starts), y)
    torch.cuda.synchronize()
    assert torch.equal(y, outs[2])
