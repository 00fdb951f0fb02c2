"""FvattnCache and FvattnPlan between calls, on the GPU."""
import pytest
import torch

from tests.test_cache_gpu import bf16, i32

pytestmark = pytest.mark.gpu


def test_errors_and_lengths_of_a_cache():
    import numpy as np
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(3)
    for capture in (False, True):
        c = fv.FvattnCache(2, 2, 64, 64, 256)
        K, V, Q = bf16(rng, 2, 2, 5, 64), bf16(rng, 2, 2, 5, 64), bf16(rng, 2, 2, 5, 64)
        counts = i32([5, 5])

        def step():
            c.append(K, V, new_lens=counts)
            return c.attend(Q)

        def again():
            step() if graph is None else graph.replay()

        graph = None
        step()
        c.check()
        if capture:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        again()
        c.check()
        assert c.lens.tolist() == [10, 10]
        counts.copy_(i32([6, -1]))
        again()
        assert c.lens.tolist() == [15, 10]
        counts.copy_(i32([1, 5]))
        again()
        again()
        assert c.status.tolist() == [0, 0]
        with pytest.raises(fv.FvattnError) as e:
            c.check()
        assert e.value.status == fv.FVATTN_ERR_BAD_PAGE
        c.check()
        assert c.lens.tolist() == [17, 20]
        table = c.page_table.clone()
        c.page_table[1, 0] = 99   # attention of one call meets it
        c.attend(Q)
        c.page_table.copy_(table)
        again()
        with pytest.raises(fv.FvattnError):
            c.check()
        c.check()


def test_a_plan_with_positions_allocates_nothing_more():
    import numpy as np
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(5)
    pos, axes = fv.grid_positions(4, 8, 8), fv.rope_axes((24, 20, 20))
    Q, K, V = (bf16(rng, 1, 2, 256, 64, layout=x) for x in ("bnhd", "bnhd", "bhnd"))
    plan = fv.FvattnPlan(1, 2, 256, 64, 64)
    O = plan(Q, K, V, 0.9, positions=pos, rope=axes)[0].clone()
    turned = [t.clone() for t in plan.turned]
    plan(K, Q, V, 0.9, positions=pos, rope=axes)
    torch.cuda.synchronize()
    before, at = torch.cuda.memory_allocated(), [t.data_ptr() for t in plan.turned]
    torch.cuda.reset_peak_memory_stats()
    again = plan(Q, K, V, 0.9, positions=pos, rope=axes)[0]
    plan.check()
    assert torch.cuda.max_memory_allocated() == before and [t.data_ptr() for t in plan.turned] == at
    assert torch.equal(again, O) and all(torch.equal(a, b) for a, b in zip(plan.turned, turned))
    s = torch.cuda.Stream()
    plan.O.zero_()
    s.wait_stream(torch.cuda.current_stream())
    plan(Q, K, V, 0.9, positions=pos, rope=axes, stream=s)
    s.synchronize()
    assert torch.equal(plan.O, O)
