"""One zero-filled workspace for beam selection and the fused decodes of a step, in turn and in graphs: each call's results
are those on a workspace of its own, bit for bit."""
import pytest
import torch

from test_gpu_beam import DEV, DT, I32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("graphed", [False, True])
def test_selections_and_decodes_on_one_workspace(lib, graphed):
    g = torch.Generator(device=DEV).manual_seed(4)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)
    calls, sizes = [], []
    for B, K, V, M, dtype in [(3, 4, 32000, 8, "f32"), (64, 2, 999, 4, "bf16"), (1, 16, 50257, 32, "bf16")]:
        logits, scores = (2 * normal(B, K, V)).to(DT[dtype]), normal(B, K)
        calls.append(lambda ws, a=(logits, scores), M=M: lib.cp_beam_select(*a, num_candidates=M, eos_token=1, workspace=ws))
        sizes.append(lib.cp_beam_select_workspace_size(B, K, V, M))
    for kind, B, Hq, Hkv, d, L in [("bf16", 6, 8, 2, 64, 700), ("q4", 2, 8, 8, 128, 3000), ("f32", 30, 4, 1, 128, 333)]:
        cp, I, cols = 2, 8, -(-L // 32) + 1
        pool = B * cols
        if kind == "q4":        # records that rows were written to
            kc, vc = (torch.zeros(cp, pool, Hkv, 9 * d, dtype=torch.uint8, device=DEV) for _ in range(2))
        else:
            kc, vc = (torch.zeros(cp, pool, Hkv, 16, d, dtype=DT[kind], device=DEV) for _ in range(2))
        dt = DT["f32" if kind == "f32" else "bf16"]
        tables = torch.arange(pool, **I32).view(1, B, cols).expand(cp, -1, -1).contiguous()
        x = normal(B * L, 2 * Hkv, d).to(dt)
        lib.cp_rope_kv_cache_write(x[:, :Hkv], x[:, Hkv:], torch.arange(B + 1, **I32) * L, torch.zeros(B, **I32), kc, vc, tables, cp, I)
        q, lens = normal(B, Hq, d).to(dt), torch.randint(L // 2, L + 1, (B,), generator=g, device=DEV).int()
        names = ("cp_decode_attention_q4",) if kind == "q4" else ("cp_decode_attention", "cp_decode_attention_mod")
        for name in names:
            calls.append(lambda ws, f=getattr(lib, name), a=(q, kc, vc, tables, lens, cp, I), L=L:
                         f(*a, max_seq_len=L, workspace=ws))
        sizes.append(lib.cp_decode_workspace_size(B, Hq, Hkv, d, cp, 64))
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device=DEV)
    want = [[t.clone() for t in f(torch.zeros(max(sizes), dtype=torch.uint8, device=DEV))] for f in calls]
    torch.cuda.synchronize()
    order = [i for step in range(1, len(calls)) for i in range(0, step * len(calls), step)]
    if not graphed:
        for i in order:
            assert all(torch.equal(a, b) for a, b in zip(calls[i % len(calls)](ws), want[i % len(calls)])), i
    else:
        graphs = []
        for f in calls:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs = f(ws)
            graphs.append((graph, outs))
        for i in order:
            graph, outs = graphs[i % len(calls)]
            for t in outs:
                t.fill_(-3)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i % len(calls)])), i
    torch.cuda.synchronize()
    assert int(ws[:65536 * 4].view(torch.int32).abs().max()) == 0
