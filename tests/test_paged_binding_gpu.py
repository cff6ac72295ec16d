"""The paged cache's calls as a serving loop makes them: steps without rows."""
import pytest
import torch

from test_paged_gpu import api, attn_case, i32, shape_config  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_step_without_rows(api):
    """Two sequences end and a third is idle: the plan has no rows, and the
    step's other calls take them, with and without a workspace."""
    cfg = shape_config(8, 2, 64)
    c = attn_case(2, 8, 2, 64, 16, 20, [9, 5, 3], [0, 0, 0])
    table, before = i32(c["table"]), (c["k"].clone(), c["v"].clone())
    n_pages = c["k"].shape[0]
    queue, state = i32(list(range(n_pages))), i32([0, 0])
    ws = api.zeros_workspace(256)
    p = api.paged_plan(i32([-1, 0, -1]), i32([9, 5, 3]), state, queue, table, 16, 0, prefix_len=20, ws=ws)
    api.check(ws)
    assert p.lens.tolist() == [0, 5, 0] and p.row_start.tolist() == [0] * 4 and p.slots.shape == p.pos.shape == (0,)
    assert p.state.tolist() == [0, 2]
    for w in (ws, None):
        q = api.qk_prep_paged(cfg, True, torch.empty((0, cfg.qkv_dim), device="cuda"), torch.ones(512, device="cuda"),
                              torch.ones(128, device="cuda"), p.pos, p.slots, c["k"], c["v"], ws=w)
        assert q.shape == (0, 8, 64) and q.dtype == torch.bfloat16
        out = api.attn_shared(q, c["k"], c["v"], p.row_start, p.lens, table, i32(c["ptab"]), 20, max_new=1, ws=w)
        assert out.shape == (0, 8, 64) and out.dtype == torch.bfloat16
    assert api.attn_shared_workspace(0, 3, 8, 2, 64).numel() >= 256
    torch.cuda.synchronize()
    assert torch.equal(c["k"], before[0]) and torch.equal(c["v"], before[1])
    # the other arguments are checked all the same
    with pytest.raises(ValueError):
        api.attn_shared(q, c["k"], c["v"], p.row_start, p.lens[:-1], table, i32(c["ptab"]), 20)
    with pytest.raises(ValueError):
        api.qk_prep_paged(cfg, True, torch.empty((0, cfg.qkv_dim), device="cuda"), torch.ones(511, device="cuda"),
                          torch.ones(128, device="cuda"), p.pos, p.slots, c["k"], c["v"])


@pytest.mark.parametrize("P,pad", [(20, 1), (5000, 1), (5000, 70), (0, 300)])
def test_rows_of_padding_alone(api, P, pad):
    """No sequence has a row: nothing is written, nothing reported."""
    c = attn_case(3, 8, 2, 64, 16, P, [9, 5, 300], [0, 0, 0], pad=pad)
    ws = api.attn_shared_workspace(pad, 3, 8, 2, 64, 40)
    out = torch.full_like(c["q"], 9.0)
    api.attn_shared(c["q"], c["k"], c["v"], i32(c["start"]), i32(c["lens"]), i32(c["table"]),
                    i32(c["ptab"]) if P else None, P, max_new=40, ws=ws, out=out)
    api.check(ws)
    assert torch.all(out == 9.0)


def test_a_plan_keeps_its_error_word(api):
    """Without a workspace of the caller's the plan's own holds the error word;
    it serves the append too."""
    from w4_weight_only_b200 import _abi
    args = (i32([0]), i32([0, 1]), i32([0]), i32([[-1, -1]]), 16, 32)
    good = api.paged_plan(i32([16]), *args)
    api.check(good.ws)
    assert good.lens.tolist() == [16] and len(good) == 5
    fails = api.paged_plan(i32([17]), *args)  # two pages of one
    assert fails.lens.tolist() == [0] and fails.slots.tolist() == [-1] * 32
    with pytest.raises(_abi.W4AError) as e:
        api.check(fails.ws)
    assert e.value.code == _abi.ERR_KERNEL
    api.check(good.ws)  # its own
    ws = api.zeros_workspace(256)
    out = api.PagedPlan(*(torch.empty_like(t) for t in good))
    again = api.paged_plan(i32([16]), *args, ws=ws, out=out)
    assert again.ws is ws and all(a is b for a, b in zip(again, out))
    for a, b in zip(again, good):
        assert torch.equal(a, b)
    cfg = shape_config(8, 2, 64)
    k = torch.zeros((1, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.ones((32, cfg.qkv_dim), device="cuda")
    bad = good.slots.clone()
    bad[3] = 16
    gains = torch.ones(512, device="cuda"), torch.ones(128, device="cuda")
    api.qk_prep_paged(cfg, True, y, *gains, good.pos, good.slots, k, k.clone(), ws=good.ws)
    api.check(good.ws)
    api.qk_prep_paged(cfg, True, y, *gains, good.pos, bad, k, k.clone(), ws=good.ws)
    with pytest.raises(_abi.W4AError):
        api.check(good.ws)


def test_one_workspace_for_a_step(api):
    """The attention's workspace serves the three calls of a step, and one check
    covers them; only its first 256 bytes have to be zero."""
    from w4_weight_only_b200 import _abi
    cfg, B, P = shape_config(8, 2, 64), 3, 40
    c = attn_case(4, 8, 2, 64, 16, P, [30, 18, 2], [1, 1, 1])
    good = api.attn_shared(c["q"], c["k"], c["v"], i32(c["start"]), i32(c["lens"]), i32(c["table"]), i32(c["ptab"]), P)
    ws = api.attn_shared_workspace(B, B, 8, 2, 64)
    assert not ws[:256].any()
    ws[256:] = 255
    n = c["k"].shape[0]
    step = dict(state=i32([0, 0]), queue=i32([0] * n), table=i32(c["table"]), page_size=16, max_rows=B, prefix_len=P, ws=ws)
    p = api.paged_plan(i32([1] * B), i32([x - 1 for x in c["lens"]]), **step)
    y = torch.randn((B, cfg.qkv_dim), device="cuda")
    k, v = c["k"].clone(), c["v"].clone()
    api.qk_prep_paged(cfg, True, y, torch.ones(512, device="cuda"), torch.ones(128, device="cuda"), p.pos, p.slots, k, v,
                      ws=ws)
    out = api.attn_shared(c["q"], c["k"], c["v"], p.row_start, p.lens, i32(c["table"]), i32(c["ptab"]), P, ws=ws)
    api.check(ws)
    assert torch.equal(out, good)
    api.paged_plan(i32([1] * B), i32([x + 60 for x in c["lens"]]), **step)  # beyond the table
    with pytest.raises(_abi.W4AError):
        api.check(ws)
