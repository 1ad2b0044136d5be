"""The attention half of the verify forward together with verification and
commit, as a decoding loop uses them: prompts, rounds of drafted trees, the
commit, the next round.  A one-layer model with random weights in float32;
the emitted tokens must be those of decoding one token at a time with the
whole prefix recomputed in float64."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_verification_04_amd as sv
import workloads as W
from tests._gpu import DEV, commit, compact_tree, commit_paged, i32, note, requires_gpu, verify_tree, verify_greedy

pytestmark = [pytest.mark.gpu, requires_gpu]

H, G, D, V, EPS = 2, 2, 32, 50, 1e-5
FREQ = (100.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)


class Model:
    def __init__(self, seed):
        r = np.random.default_rng(seed)
        self.emb = r.standard_normal((V, (G + 2) * H, D)).astype(np.float32)      # token -> q, k, v
        self.head = r.standard_normal((H * G * D, V)).astype(np.float32)
        self.wq, self.wk = (1 + 0.3 * r.standard_normal((2, D))).astype(np.float32)
        self.dev = [torch.from_numpy(x).to(DEV) for x in (self.emb, self.head, self.wq, self.wk, FREQ)]

    def next_token(self, tokens):
        """Greedy continuation in float64, and the two largest logits' distance."""
        x = self.emb[np.array(tokens)].astype(np.float64)
        p = np.arange(len(tokens))
        q = oracle.norm_rope(x[:, :H * G], self.wq, EPS, p, FREQ)[-1]
        k = oracle.norm_rope(x[:, H * G:H * G + H], self.wk, EPS, p, FREQ)
        v = x[:, H * G + H:]
        o = np.concatenate([oracle.attend(q[j:j + 1], k[:, j // G], v[:, j // G], np.ones((1, len(tokens)), bool),
                                          D ** -0.5)[0][0] for j in range(H * G)])
        z = np.sort(o @ self.head.astype(np.float64))
        assert z[-1] - z[-2] > 1e-3                        # no tie that float32 could turn
        return int(np.argmax(o @ self.head.astype(np.float64)))

    def qkv(self, tokens):
        x = self.dev[0][torch.as_tensor(np.asarray(tokens), device=DEV).long()]
        return x[..., :H * G, :], x[..., H * G:H * G + H, :], x[..., H * G + H:, :]

    def norms(self):
        return dict(q_weight=self.dev[2], k_weight=self.dev[3], eps=EPS, inv_freq=self.dev[4])


def _prompt(model, prompts, kv, where, paged):
    """Rows of all tokens but each prompt's last (it has no KV yet); returns the
    prompts' attention, packed."""
    lens = np.array([len(p) - 1 for p in prompts])
    cu, n = i32(np.concatenate([[0], np.cumsum(lens)])), i32(lens)
    q, k, v = model.qkv(np.concatenate([p[:-1] for p in prompts]))
    rot = torch.empty(q.shape, device=DEV)
    f, a = ((sv.spec_norm_rope_kv_paged, sv.spec_prompt_attention_paged) if paged else
            (sv.spec_norm_rope_kv, sv.spec_prompt_attention))
    f(q, k, v, kv, 0, where, n, rot, cu_seqlens=cu, **model.norms())
    out = torch.empty_like(rot)
    a(rot, kv, 0, cu, where, n, out)
    return out, lens


def _grown(model, prompts, rounds_tokens):
    """Each sequence decoded one token at a time to the given lengths."""
    seqs = [list(p) for p in prompts]
    for s, upto in zip(seqs, rounds_tokens):
        while len(s) < upto:
            s.append(model.next_token(s))
    return seqs


def _check_prompt(model, prompts, out):
    """The logits after each prompt's rows continue it as the model does alone."""
    at = 0
    for p in prompts:
        z = out[at:at + len(p) - 1].reshape(len(p) - 1, -1) @ model.dev[1]
        for i in (0, (len(p) - 2) // 2, len(p) - 2):
            assert int(z[i].argmax()) == model.next_token(p[:i + 1])
        at += len(p) - 1


def test_tree_rounds_on_a_rectangle_equal_decoding_alone():
    rng = np.random.default_rng(0)
    model = Model(1)
    prompts = [rng.integers(0, V, x).tolist() for x in (9, 30, 2, 17)]
    B, N, rounds = 4, 12, 5
    E = max(len(p) - 1 for p in prompts)
    C = E + N * rounds + 4
    kv = torch.full((1, 2, B, H, C, D), float("nan"), device=DEV)
    note("forward: prompts")
    out, lens = _prompt(model, prompts, kv, i32([E]), False)
    _check_prompt(model, prompts, out)
    E_d, n_d = i32([E]), i32(lens)
    done = [list(p) for p in prompts]
    longest = 0
    for r in range(rounds):
        # trees whose first branches follow the model for a while
        fc, ns, draft = np.full((B, N), -1, np.int32), np.full((B, N), -1, np.int32), np.zeros((B, N), np.int32)
        for b in range(B):
            parent, fc[b], ns[b] = W.random_tree(rng, N, 3)
            text = {0: done[b]}
            for i in range(1, N):
                before = text[int(parent[i])]
                draft[b, i] = model.next_token(before) if rng.random() < 0.6 else rng.integers(0, V)
                text[i] = before + [int(draft[b, i])]
            draft[b, 0] = done[b][-1]
        fcd, nsd = i32(fc), i32(ns)
        pos = torch.empty(B, N, dtype=torch.int32, device=DEV)
        bits = torch.empty(B, N, 1, dtype=torch.int32, device=DEV)
        note(f"forward: round {r}")
        sv.spec_tree_mask(fcd, nsd, n_d, pos, bits)
        q, k, v = model.qkv(draft)
        rot, att = torch.empty(q.shape, device=DEV), torch.empty(q.shape, device=DEV)
        sv.spec_norm_rope_kv(q, k, v, kv, 0, E_d, n_d, rot, positions=pos, **model.norms())
        ws = sv.workspace(sv.spec_tree_attention_workspace_bytes(B, N, H, G, D, C, sv.SPEC_F32), DEV)
        sv.spec_tree_attention(rot, kv, 0, E_d, n_d, att, ws, mask=bits)
        logits = (att.reshape(B * N, -1) @ model.dev[1]).view(B, N, V)
        got = verify_tree(logits, i32(draft), fcd, nsd)
        compact_tree(kv, N, E_d, got["path"], got["emit_count"])
        c = commit(kv, N - 1, E_d, n_d, got["emit_count"])
        E_d, n_d = c["end_col"], c["kv_len"]
        emit, toks = got["emit_count"].cpu().numpy(), got["out_tokens"].cpu().numpy()
        for b in range(B):
            done[b] += [int(x) for x in toks[b][:emit[b]]]
        longest = max(longest, int(emit.max()))
    assert done == _grown(model, prompts, [len(s) for s in done]) and longest >= 3


@pytest.mark.parametrize("page", [4, 64])
def test_linear_rounds_on_pages_equal_decoding_alone(page):
    """page 64: one page per sequence, as the ragged pool of the same-length scheduler has them."""
    rng = np.random.default_rng(2)
    model = Model(3)
    prompts = [rng.integers(0, V, x).tolist() for x in (5, 12, 2)]
    B, k, rounds = 3, 3, 5
    per = -(-64 // page)
    order = rng.permutation(B * per).reshape(B, per).astype(np.int32)
    table = i32(order)
    pool = torch.full((1, 2, B * per, H, page, D), float("nan"), device=DEV)
    note("forward: paged prompts")
    out, lens = _prompt(model, prompts, pool, table, True)
    _check_prompt(model, prompts, out)
    n_d = i32(lens)
    done = [list(p) for p in prompts]
    for r in range(rounds):
        draft = np.zeros((B, k), np.int32)
        for b in range(B):
            text = list(done[b])
            for j in range(k):
                draft[b, j] = model.next_token(text) if rng.random() < 0.7 else rng.integers(0, V)
                text.append(int(draft[b, j]))
        slots = np.concatenate([np.array([[s[-1]] for s in done]), draft], 1)
        q, kk, v = model.qkv(slots)
        rot, att = torch.empty(q.shape, device=DEV), torch.empty(q.shape, device=DEV)
        note(f"forward: paged round {r}")
        sv.spec_norm_rope_kv_paged(q, kk, v, pool, 0, table, n_d, rot, **model.norms())
        ws = sv.workspace(sv.spec_tree_attention_workspace_bytes(B, k + 1, H, G, D, per * page, sv.SPEC_F32), DEV)
        sv.spec_tree_attention_paged(rot, pool, 0, table, n_d, att, ws)
        logits = (att.reshape(B * (k + 1), -1) @ model.dev[1]).view(B, k + 1, V)
        got = verify_greedy(logits, i32(draft))
        n_d = commit_paged(k, page, n_d, got["emit_count"], table)["kv_len"]
        emit, toks = got["emit_count"].cpu().numpy(), got["out_tokens"].cpu().numpy()
        for b in range(B):
            done[b] += [int(x) for x in toks[b][:emit[b]]]
    assert done == _grown(model, prompts, [len(s) for s in done])
