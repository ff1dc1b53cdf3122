"""A whole speculative cycle through the public calls: context appended, a
block drafted, the target's cache written, its attention, its logits adjusted,
the block verified, lengths and counts moved on; against the oracle's parts,
and eager against one captured graph."""

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from block_speculative_decoding_ctx_gb300 import synth
from oracle import target as ot
from oracle import verify as over
from test_gpu_target_chain import Target
from target_testutil import F8, to64

pytestmark = pytest.mark.gpu
B, GAMMA = 3, 4


class Cycle:
    def __init__(self, e4m3):
        dims = synth.DIMS["tiny"]
        V, dev = dims["vocab"], "cuda"

        def put(x):
            if isinstance(x, dict):
                return {k: put(v) for k, v in x.items()}
            return [put(v) for v in x] if isinstance(x, list) else x.to(dev)
        self.h = dfl.dflash_create(dict(
            hidden=dims["d"], n_q_heads=dims["n_q"], n_kv_heads=dims["n_kv"], head_dim=dims["hd"], ffn=dims["ffn"], vocab=V,
            n_layers=dims["n_layers"], n_feat=dims["n_feat"], feat_dim=dims["feat_dim"], window=dims["window"], gamma_max=GAMMA,
            topk_max=4, batch_max=B, append_max=GAMMA, rope_theta=1.0e6, eps=1.0e-6, mask_id=-1),
            put(synth.weights(dims, 3, random_gains=True)))
        self.feats = synth.features(dims, B * GAMMA, 4).reshape(B, GAMMA, dims["n_feat"], dims["feat_dim"]).to(dev)
        ring = (dims["n_layers"], B, dims["n_kv"], dims["window"], dims["hd"])
        self.rk, self.rv = (torch.zeros(ring, dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.ctx = torch.zeros(B, dtype=torch.int64, device=dev)
        self.n_app = torch.tensor([3, 1, 4], dtype=torch.int32, device=dev)
        self.anchor = torch.tensor([5, 7, 11], dtype=torch.int32, device=dev)
        self.block = torch.empty(B, GAMMA - 1, dtype=torch.int32, device=dev)
        self.logits = torch.empty(B, GAMMA - 1, V, device=dev)
        self.ws_a = dfl.workspace(dfl.dflash_append_workspace_bytes(self.h))
        self.ws_d = dfl.workspace(dfl.dflash_draft_workspace_bytes(self.h))
        self.t = Target(B, GAMMA, V, n_q=6, n_kv=2, hd=64, page=16, pages=30, e4m3=e4m3, seed=3, lens=[40, 5, 100])
        # the first and third request favour what was drafted, so that some of it is accepted
        self.t.pen.update(bias_start=torch.tensor([0, GAMMA - 1, GAMMA - 1, 2 * (GAMMA - 1)], dtype=torch.int32, device=dev),
                          bias_ids=torch.zeros(2 * (GAMMA - 1), dtype=torch.int32, device=dev),
                          bias_vals=torch.full((2 * (GAMMA - 1),), 50.0, device=dev))
        self.t.allow.fill_(-1)

    def run(self):
        t = self.t
        dfl.dflash_ctx_append(self.h, self.feats, self.n_app, self.ctx, self.rk, self.rv, self.ws_a)
        dfl.dflash_draft_block(self.h, self.anchor, self.ctx, self.rk, self.rv, GAMMA, self.ws_d, topk=0,
                               out=dict(logits=self.logits, draft=self.block))
        t.tokens_in[:, 0] = self.anchor
        t.tokens_in[:, 1:] = self.block
        t.draft.copy_(self.block)
        t.pen["bias_ids"].copy_(torch.cat([self.block[0], self.block[2]]))
        t.step()

    def move_on(self):
        t = self.t
        ok = t.tokens >= 0
        t.counts.scatter_add_(1, t.tokens.clamp(min=0).long(), ok.to(torch.int32))
        t.kv_len += t.n_append.long()
        self.anchor.copy_(t.anchor)
        self.n_app.copy_(t.n_append)

    def tensors(self):
        t = self.t
        mine = [self.rk, self.rv, self.ctx, self.n_app, self.anchor, self.block, t.kv_len, t.counts, t.tokens, t.accept,
                t.out, t.adjusted, t.pages.view(torch.uint8) if t.pages.dtype is F8 else t.pages]
        return mine + ([] if t.scale[0] is None else [t.scale])

    def statuses(self):
        return [dfl.dflash_read_status(w) for w in (self.ws_a, self.ws_d, self.t.ws, self.t.ws_v)]


@pytest.mark.parametrize("e4m3", [False, True])
def test_cycles_of_drafter_and_target_eager_and_captured(e4m3):
    eager = Cycle(e4m3)
    history, accepted = [], 0
    for _ in range(4):
        counts = eager.t.counts.cpu().numpy()
        eager.run()
        torch.cuda.synchronize()
        t = eager.t
        assert eager.statuses() == [0, 0, 0, 0]
        draft = eager.block.cpu().numpy()
        np.testing.assert_array_equal(draft, eager.logits.argmax(-1).cpu().numpy())
        par = {k: t.pen[k].cpu().numpy() for k in ("repetition", "frequency", "presence")}
        bias = [(b, int(v), 50.0) for b in (0, 2) for v in draft[b]]
        want, size = ot.adjust(to64(t.logits), counts=counts, draft=draft, bias=bias, **par)
        # a quotient's, a product's and three sums' roundings, and a sum per bias of an id
        assert (np.abs(to64(t.adjusted) - want) <= (6 + GAMMA) * 2.0 ** -24 * size).all()
        n, tok = over.greedy(t.adjusted.cpu().numpy(), draft)
        np.testing.assert_array_equal(t.accept.cpu().numpy(), n)
        np.testing.assert_array_equal(t.tokens.cpu().numpy(), tok)
        np.testing.assert_array_equal(t.n_append.cpu().numpy(), n + 1)
        accepted += int(n.sum())
        eager.move_on()
        torch.cuda.synchronize()
        history.append([x.clone() for x in eager.tensors()])
    assert accepted > 0

    warm, graphed, fresh = Cycle(e4m3), Cycle(e4m3), Cycle(e4m3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        warm.run()
        warm.move_on()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        graphed.run()
        graphed.move_on()
    for a, b in zip(graphed.tensors(), fresh.tensors()):
        a.copy_(b)
    torch.cuda.synchronize()
    for want in history:
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(graphed.tensors(), want):
            assert torch.equal(a, b)
    assert graphed.statuses() == [0, 0, 0, 0]
