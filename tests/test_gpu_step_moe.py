"""The composed draft-and-verify step with a target whose layers 1, 2 and 4 are mixtures of three
experts (layers 0 and 3 stay dense, so that folded and unfolded norms meet on both sides), against
the oracle.  Every row takes all three experts, with softmax weights of the router's logits: the
layer is then a continuous function of its input, and the bf16 tolerance of the dense step's test
applies (a chosen subset could change at a near tie).  The choice of a subset is tested exactly in
test_gpu_moe.py."""
import numpy as np
import pytest
import torch

import eagle_tree_speculative_spec_gb300 as e3
import synth
from oracle import accept as oacc
from tests import test_gpu_step as dense
from tests._util import require_gpu

pytestmark = pytest.mark.gpu

MOE_LAYERS, E, FE = (1, 2, 4), 3, 160


def _build(dev, fold):
    st, t_f, d_f = dense._build(dev, oacc.TOPK, fold_norms=fold)
    d = dense.CFG["d"]
    r = synth.rng(29, 1)
    st.target["router"] = [None] * dense.CFG["layers"]
    for l in MOE_LAYERS:
        for name, key, shape, scale in (("wg", "w_gate", (E, FE, d), d ** -0.5), ("wu", "w_up", (E, FE, d), d ** -0.5),
                                        ("wd", "w_down", (E, d, FE), 0.5 * FE ** -0.5), ("router", "router", (E, d), d ** -0.5)):
            gpu, ref = synth.to_bf16(scale * r.standard_normal(shape, dtype=np.float32))
            st.target[name][l] = gpu.to(dev)
            t_f[f"layers.{l}.{key}"] = ref
    st.cfg.update(experts_per_token=E)
    st._folded = None
    st.prepare(ws_linear_bytes=64 << 20, ws_attn_bytes=16 << 20)
    target = dense._oracle_target(t_f)
    target.moe = dict(k=E)
    return st, target


@pytest.mark.parametrize("fold", [False, True])
def test_moe_step_matches_oracle(fold):
    dev = require_gpu()
    st, target = _build(dev, fold)
    for step in range(2):
        before = {k: v.float().cpu().numpy() if v.dtype == torch.bfloat16 else v.cpu().numpy()
                  for k, v in dense._snapshot(st).items()}
        st.run()
        torch.cuda.synchronize()
        g = dense._host(st)
        assert g["dev_status"][0] == 0
        dense._check_verify(target, before, g)
        dense._check_accept_and_compact(oacc.TOPK, before, g, step)


def test_moe_step_graph_replay_and_subset():
    """Two of the three experts: the replayed graph gives the eager step's bits; and flops() counts the
    experts taken."""
    dev = require_gpu()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        st, _ = _build(dev, True)
        all_flops = st.flops()[0]
        st.cfg.update(experts_per_token=2, moe_scoring=e3.MOE_SIGMOID)
        st.prepare(ws_linear_bytes=64 << 20, ws_attn_bytes=16 << 20)
        rows = dense.CFG["B"] * dense.CFG["N"]
        assert all_flops - st.flops()[0] == len(MOE_LAYERS) * 2 * rows * 3 * dense.CFG["d"] * FE
        snap = dense._snapshot(st)
        st.run()
        torch.cuda.synchronize()
        eager = dense._host(st)
        dense._restore(st, snap)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            st.run()
        dense._restore(st, snap)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = dense._host(st)
    assert int(st.dev_status) == 0
    for k in eager:
        assert np.array_equal(eager[k], replayed[k]), k


def test_moe_shapes_are_checked():
    dev = require_gpu()
    st, _ = _build(dev, False)
    st.target["wd"][2] = st.target["wd"][2][:, :, :32].contiguous()
    with pytest.raises(ValueError, match="wd"):
        st.prepare(ws_linear_bytes=64 << 20, ws_attn_bytes=16 << 20)
