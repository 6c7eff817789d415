"""Calls on two streams at once, each with its own workspace and outputs, give what they give alone: window attention and the
8-bit cache beside each other and beside the calls over bf16 pages that hold tensor memory too."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BK, D = 128, 128


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def work(msa, seed):
    """Inputs, and [(what fills its outputs, the outputs)] of one stream."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    Hkv, G, per = 4, 6, 12
    P, lengths, calls = 5 * per, [1500, 700, 129, 1, 1400], []
    K, V = rand(P, Hkv, BK, D), rand(P, Hkv, BK, D)
    pt, L = torch.randperm(P, generator=g, device="cuda").int().view(5, per), i32(lengths)
    cache = msa.q8_cache(P, Hkv, "cuda")
    msa.msa_cache_append_q8(K.transpose(1, 2).reshape(-1, Hkv, D), V.transpose(1, 2).reshape(-1, Hkv, D),
                            torch.arange(P * BK, device="cuda"), cache)
    new = lambda *s: (torch.empty(*s, D, dtype=torch.bfloat16, device="cuda"), torch.empty(*s, device="cuda"))  # noqa: E731

    def add(f, *out):
        calls.append((lambda s: f(s, *out), out))

    Q = rand(5, Hkv * G, D)
    for B, S in ((1, 900), (2, 30), (5, 4)):     # many tiles, few, and few over pages
        q = rand(B, S, Hkv * G, D)
        if S > 4:
            k, v = rand(B, S, Hkv, D), rand(B, S, Hkv, D)
            add(lambda s, O, E, q=q, k=k, v=v: msa.msa_window_attn_prefill(q, k, v, O, E, window=300, sinks=4, stream=s), *new(B, S, Hkv * G))
        else:
            pos = L - S + 3
            add(lambda s, O, E, q=q, pos=pos: msa.msa_window_attn_prefill(
                q, K, V, O, E, window=300, sinks=4, seq_pt=pt, q_pos=pos.clamp(min=0), stream=s), *new(B, S, Hkv * G))
    ws = [torch.zeros(msa.msa_attn_decode_q8_workspace_size(5, Hkv), dtype=torch.uint8, device="cuda") for _ in range(3)]
    add(lambda s, O, E: msa.msa_window_attn_decode(Q, K, V, pt, L, O, E, ws[0], window=1 << 30, stream=s, scratch_zeroed=True), *new(5, Hkv * G))
    add(lambda s, O, E: msa.msa_dense_attn_decode_q8(Q, cache, pt, L, O, E, ws[1], stream=s, scratch_zeroed=True), *new(5, Hkv * G))
    few, n, last = pt[:, None, :8].expand(5, Hkv, 8).reshape(5 * Hkv, 8).contiguous(), i32([8, 3, 0, 1] * 5), i32([77] * 20)
    add(lambda s, O, E: msa.msa_sparse_attn_decode_q8(Q, cache, few, n, last, O, E, ws[2], stream=s, scratch_zeroed=True), *new(5, Hkv * G))
    add(lambda s, *o: msa.msa_cache_expand_q8(cache, pt.flatten(), *o, stream=s),
        *(torch.empty(P, Hkv, BK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    to = torch.empty(2 * P, Hkv, BK, D, dtype=torch.bfloat16, device="cuda")
    to[:P] = K
    src, dst = torch.arange(P, dtype=torch.int32, device="cuda"), torch.arange(P, 2 * P, dtype=torch.int32, device="cuda")
    add(lambda s, o: msa.msa_copy_pages([o], src, dst, stream=s), to)
    q, k, v = rand(1, 700, Hkv * G, D), rand(1, 700, Hkv, D), rand(1, 700, Hkv, D)
    add(lambda s, O, E: msa.msa_dense_attn_prefill(q, k, v, O, E, stream=s), *new(1, 700, Hkv * G))
    return calls


def test_two_streams(msa):
    sides = [work(msa, seed) for seed in (21, 22)]
    want = []
    for calls in sides:
        for f, _ in calls:
            f(None)
        torch.cuda.synchronize()
        want.append([[o.clone() for o in out] for _, out in calls])
    streams = [torch.cuda.Stream() for _ in sides]
    for shift in range(len(sides[0])):           # each call beside every other one
        for calls in sides:
            for _, out in calls:
                for o in out:
                    if o.dim() != 4 or o.shape[0] != 120:
                        o.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for j in range(len(sides[0])):
                for side, (calls, s) in enumerate(zip(sides, streams)):
                    calls[(j + shift * side) % len(calls)][0](s)
        torch.cuda.synchronize()
        for calls, w in zip(sides, want):
            for (_, out), x in zip(calls, w):
                for a, b in zip(out, x):
                    assert torch.equal(a, b)
