"""The serving and scoring operators used together: prompts rotated into a cache of 16-bit pages and one of 4 bits, tokens decoded
over both, logits sampled and scored; a training step through rotation and attention, and one through log probabilities.

Tolerances. Against the 16-bit cache's reference: one rounding of the rotated rows (the reference takes them from the device),
two bf16 parts of the probabilities (2^-16) and y's own rounding, 2^-8 of the value and 2^-12 of the largest value in sight. The
4-bit cache: serving_ref.attend4's bounds. Training: norms, seven roundings to bf16 (rotated rows, probabilities, the scores'
gradient, y, dqkv twice, the loss gradient is exact) of 2^-9 of the norm each on average: 2^-9 7 = 1.4e-2.
"""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_ref  # noqa: E402
import serving_ref as ref  # noqa: E402
from gpu_util import dev_bf16, dev_i32, host, rand_bf16  # noqa: E402

H, HKV, D, PAGE = 8, 2, 64, 16
ROW = (H + 2 * HKV) * D


class Caches:
    """Both caches of three sequences, and what the device made of their prompts."""

    def __init__(self, seed=0, counts=(40, 7, 33), T=40):
        from decoder_only_transformer_gpt_gb300 import binding
        rng = np.random.default_rng(seed)
        B = len(counts)
        self.B, self.counts = B, np.array(counts)
        self.turns = binding.rotary_turns(ref.freqs(D))
        self.table_h = rng.permutation(B * 5 + 2)[: B * 5].reshape(B, 5)
        self.table = dev_i32(self.table_h)
        n = B * 5 + 2
        self.pool = torch.zeros(n, 2, HKV, PAGE, D, dtype=torch.bfloat16, device="cuda")
        self.codes = torch.zeros(n, 2, HKV, PAGE, D // 2, dtype=torch.uint8, device="cuda")
        self.ranges = torch.zeros(n, 2, HKV, PAGE, 2, dtype=torch.bfloat16, device="cuda")
        x = dev_bf16(rand_bf16(rng, (B, T, ROW)))
        self.rows, self.rows4 = torch.zeros_like(x), torch.zeros_like(x)
        a = dict(turns=self.turns, count=dev_i32(self.counts))
        binding.paged_append(x, self.pool, self.table, H, out=self.rows, **a)
        binding.paged_append4(x, self.codes, self.ranges, self.table, H, out=self.rows4, **a)
        self.lens = dev_i32(self.counts)
        self.x = x


def test_prompts_decoding_and_scores(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    c = Caches()
    assert torch.equal(c.rows, c.rows4)
    want, mag = ref.rotate(host(c.x).reshape(c.B, 40, -1, D), H, HKV, ref.freqs(D), np.zeros(c.B), False)
    got = host(c.rows).reshape(want.shape)
    for b, n in enumerate(c.counts):
        assert (np.abs(got - want)[b, :n] <= 2.0 ** -8 * np.abs(want[b, :n]) + 5e-7 * mag[b, :n]).all()
    # the prompts' attention reads the rotated rows
    y = torch.zeros(c.B, 40, H * D, dtype=torch.bfloat16, device="cuda")
    binding.attention_window(c.rows, y, H, HKV, window=40)
    last = got[0, 39]
    for h in (0, 7):
        k, u = got[0, :, H + h // 4], got[0, :, H + HKV + h // 4]
        w = paged_ref.attend(last[h], k, u)[0]
        assert (np.abs(host(y)[0, 39].reshape(H, D)[h] - w) <= 2.0 ** -8 * np.abs(w) + 2.0 ** -8 * np.abs(u).max()).all()
    # tokens: rotation and store, then the attention; the 4-bit side as one graph that counts the lengths up
    new, rows = torch.zeros(c.B, 1, ROW, dtype=torch.bfloat16, device="cuda"), torch.zeros(c.B, 1, ROW, dtype=torch.bfloat16, device="cuda")
    rows4, y4 = torch.zeros_like(rows), torch.zeros(c.B, H * D, dtype=torch.bfloat16, device="cuda")
    y16, lse4, lens4 = torch.zeros_like(y4), torch.zeros(c.B, H, device="cuda"), c.lens.clone()

    def token4():
        binding.paged_append4(new, c.codes, c.ranges, c.table, H, turns=c.turns, start=lens4, out=rows4)
        binding.paged_attention4(rows4[:, 0], c.codes, c.ranges, c.table, lens4, y4, H, lse2=lse4, added=1)
    kept = c.codes.clone(), c.ranges.clone()
    token4()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token4()
        lens4 += 1
    c.codes.copy_(kept[0])
    c.ranges.copy_(kept[1])
    rng = np.random.default_rng(3)
    for step in range(12):
        new.copy_(dev_bf16(rand_bf16(rng, (c.B, 1, ROW), 1.5)))
        binding.paged_append(new, c.pool, c.table, H, turns=c.turns, start=c.lens, out=rows)
        binding.paged_attention(rows[:, 0], c.pool, c.table, c.lens, y16, H)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rows, rows4)
        n = host(c.lens).astype(int)
        pool = host(c.pool)
        want16, _, _, _ = paged_ref.decode(host(rows)[:, 0], pool, None, c.table_h, n, H, 0, 0)
        assert (np.abs(host(y16) - want16) <= 2.0 ** -8 * np.abs(want16) + 2.0 ** -12 * np.abs(pool).max()).all()
        w4, l4, ey, el = ref.attend4(host(rows)[:, 0].astype(np.float32), c.codes.cpu().numpy(), host(c.ranges).astype(np.float32),
                                     c.table_h, n, H, 0, 0, 1)
        assert (np.abs(host(y4) - w4) <= 2.0 ** -8 * np.abs(w4) + 1.01 * ey).all() and (np.abs(host(lse4) - l4) <= el).all()
        c.lens += 1
    binding.status()
    # the rows that the 4-bit cache holds, in 16 bits: half a step of 1/15 of the row's range, its rounding and the scale's
    back = torch.zeros(c.B, 52, 2 * HKV * D, dtype=torch.bfloat16, device="cuda")
    binding.paged_load4(c.codes, c.ranges, c.table, back, count=c.lens)
    back, pool = host(back).reshape(c.B, 52, 2, HKV, D), host(c.pool)
    for b in range(c.B):
        for r in range(int(host(c.lens)[b])):
            p, s = paged_ref.place(c.table_h[b], PAGE, r)
            row = pool[p, :, :, s]
            span = row.max(-1, keepdims=True) - row.min(-1, keepdims=True)
            assert (np.abs(back[b, r] - row) <= span / 15 * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -8 * np.abs(row).max()).all()


def test_a_model_s_logits_sampled_and_scored(gpt_lib):
    import oracle
    from decoder_only_transformer_gpt_gb300 import binding
    from workloads import workload
    from workloads.generate import generate
    wl = workload("minigpt")
    w, ids, _ = generate(wl, B=3, T=24, affine="random")
    m = binding.GPTModel(wl.cfg, w, 3 * 24)
    m.kv_reserve(3)
    logits, picked = torch.zeros(3, wl.cfg.V, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    logp, entropy = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
    top_ids, top = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, device="cuda")
    m.prefill(dev_i32(ids[:, :20]), logits)
    for t in range(20, 24):
        binding.sample(logits, torch.zeros(3, device="cuda"), picked, temperature=0.0)
        binding.logprobs(logits, picked, logp, entropy=entropy, top_ids=top_ids, top_logp=top)
        assert torch.equal(top_ids[:, 0], picked) and torch.equal(top[:, 0], logp)
        a, e, i, v, _, _ = ref.logprobs(host(logits), host(picked).astype(int), 4)
        assert np.array_equal(top_ids.cpu().numpy(), i)
        # logits of a random model: differences of a few units, sums of 5,000 terms
        assert np.abs(host(logp) - a).max() <= 4e-6 and np.abs(host(entropy) - e).max() <= 8e-6 and np.abs(host(top) - v).max() <= 4e-6
        m.decode_step(dev_i32(ids[:, t]), t, logits)
    # a whole prompt's mean log probability is the model's loss
    ids_d, tg = dev_i32(ids), dev_i32(np.roll(ids, -1, 1))
    loss, full = torch.zeros(1, device="cuda"), torch.zeros(3, 24, wl.cfg.V, device="cuda")
    m.forward(ids_d, tg, loss, full)
    rows = torch.zeros(72, device="cuda")
    binding.logprobs(full.view(72, -1), tg.view(-1), rows)
    assert abs(float(rows.mean()) + float(loss)) <= 2e-5
    rloss, _ = oracle.forward(wl.cfg, w, ids, np.roll(ids, -1, 1))
    assert abs(float(rows.mean()) + rloss) <= 1e-2
    m.close()


@pytest.mark.parametrize("inter,rot", [(False, 64), (True, 32)])
def test_training_through_rotation_and_attention(gpt_lib, inter, rot):
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(6)
    B, T = 2, 75
    x, dy = rand_bf16(rng, (B, T, ROW)), rand_bf16(rng, (B, T, H * D), 0.25)
    pos = np.array([5, 90000])
    turns = binding.rotary_turns(ref.freqs(rot))
    d_x, d_dy, d_pos = dev_bf16(x), dev_bf16(dy), dev_i32(pos)
    rows, y, dqkv = torch.zeros_like(d_x), torch.zeros_like(d_dy), torch.zeros_like(d_x)
    lse2 = torch.zeros(B, H, T, device="cuda")
    binding.rotary(d_x, rows, H, HKV, turns, pos=d_pos, interleaved=inter)
    binding.attention_window(rows, y, H, HKV, window=30, sinks=2, lse2=lse2)
    binding.attention_window_bwd(rows, y, d_dy, lse2, dqkv, H, HKV, window=30, sinks=2)
    binding.rotary(dqkv, dqkv, H, HKV, turns, pos=d_pos, interleaved=inter, inverse=True)
    binding.status()
    # the same in 64 bits
    leaf = torch.from_numpy(x.astype(np.float64)).requires_grad_(True)
    v = leaf.view(B, T, H + 2 * HKV, D)
    at = torch.from_numpy(pos)[:, None].double() + torch.arange(T)
    angle = at[:, :, None, None] * torch.tensor(ref.freqs(rot), dtype=torch.float64)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    heads = v[:, :, : H + HKV]
    r = heads.clone()
    r[..., a] = heads[..., a] * angle.cos() - heads[..., b] * angle.sin()
    r[..., b] = heads[..., b] * angle.cos() + heads[..., a] * angle.sin()
    q, k, u = r[:, :, :H], r[:, :, H:].repeat_interleave(H // HKV, 2), v[:, :, H + HKV:].repeat_interleave(H // HKV, 2)
    s = torch.einsum("bthd,bshd->bhts", q, k) / D ** 0.5
    t = torch.arange(T)
    seen = (t[None] <= t[:, None]) & ((t[:, None] - t[None] < 30) | (t[None] < 2))
    out = torch.einsum("bhts,bshd->bthd", s.masked_fill(~seen, -np.inf).softmax(-1), u).flatten(2)
    out.backward(torch.from_numpy(dy.astype(np.float64)))
    for got, want in ((y, out.detach()), (dqkv, leaf.grad)):
        g, w = host(got), want.numpy()
        assert np.linalg.norm(g - w) <= 1.4e-2 * np.linalg.norm(w)


def test_training_through_log_probabilities(gpt_lib):
    # advantages and an entropy bonus, as a policy update has them; the mean of both against 64 bits
    from decoder_only_transformer_gpt_gb300 import binding
    torch.manual_seed(0)
    M, V = 37, 5003
    z = (torch.randn(M, V) * 2).cuda()
    t = torch.randint(0, V, (M,)).int().cuda()
    adv = torch.randn(M).cuda()
    lp, en, st, dz = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda"), torch.zeros(M, 2, device="cuda"), torch.zeros_like(z)
    binding.logprobs(z, t, lp, entropy=en, stats=st)
    binding.logprobs_bwd(z, t, st, adv / M, dz, entropy=en, dentropy=torch.full((M,), 0.01 / M, device="cuda"))
    leaf = z.double().requires_grad_(True)
    d = torch.distributions.Categorical(logits=leaf)
    loss = (adv.double() * d.log_prob(t.long())).mean() + 0.01 * d.entropy().mean()
    loss.backward()
    assert abs(float((adv * lp).mean() + 0.01 * en.mean()) - float(loss.detach())) <= 1e-5
    # p of 1e-4 and below, each off by 2^-20 of itself at most, and the ones of the targets by 2^-22 of dlogp
    assert float((dz.double() - leaf.grad).norm() / leaf.grad.norm()) <= 2.0 ** -19


def test_several_threads_and_streams(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    from test_gpu_paged4 import Case
    cases = [Case(8, 4, 64, 16, [700, 30, 5], seed=i, rows=r).device() for i, r in enumerate((None, 65536, None, 65536))]
    rows = [Caches(seed=i) for i in range(4)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            z = torch.randn(20, 9000, device="cuda")
            lp, en = torch.zeros(20, device="cuda"), torch.zeros(20, device="cuda")
            t = torch.arange(20, dtype=torch.int32, device="cuda")
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                for _ in range(20):
                    cases[i].call()
                    c = rows[i]
                    binding.paged_append4(c.x, c.codes, c.ranges, c.table, H, turns=c.turns, count=c.lens)
                    binding.logprobs(z, t, lp, entropy=en)
            s.synchronize()
            want = torch.log_softmax(z.double(), -1)
            if float((lp.double() - want[t.long(), t.long()]).abs().max()) > 4e-6:
                wrong.append((i, "logp"))
        except Exception as e:                       # noqa: BLE001 (shown by the main thread)
            wrong.append((i, repr(e)))
    codes = [c.codes.clone() for c in rows]
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong
    for c in cases:
        c.check()
    for c, k in zip(rows, codes):
        assert torch.equal(c.codes, k)


def test_two_graphs_with_scratch_at_once(gpt_lib):
    # each graph has scratch of its own
    from test_gpu_paged4 import Case
    cases = [Case(8, 4, 64, 16, [900, 333], seed=40 + i, rows=65536).device() for i in range(2)]
    graphs = []
    for c in cases:
        c.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_streams_given_and_refused(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    z, lp = torch.randn(4, 5000, device="cuda"), torch.zeros(4, device="cuda")
    t = torch.arange(4, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.logprobs(z, t, lp, stream=side)
    side.synchronize()
    assert torch.allclose(lp, torch.log_softmax(z, -1)[t.long(), t.long()], atol=1e-5)

    class Other:
        device_index, cuda_stream = torch.cuda.current_device() + 1, 0
    with pytest.raises(ValueError, match="stream"):
        binding.logprobs(z, t, lp, stream=Other())
    with pytest.raises(AttributeError):
        binding.logprobs(z, t, lp, stream=object())
    for bad in (z.cpu(), None, "z"):
        with pytest.raises((ValueError, TypeError)):
            binding.logprobs(bad, t, lp)
    with pytest.raises(ValueError, match="targets"):
        binding.logprobs(z, t.cpu(), lp)
    with pytest.raises(ValueError, match="logp"):
        binding.logprobs(z, t, lp[:3])


def test_calls_without_rows(gpt_lib):
    # an empty chunk of a prompt: tensors without an address
    from decoder_only_transformer_gpt_gb300 import binding
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    turns = binding.rotary_turns([10000.0 ** (-2.0 * i / 64) for i in range(32)])
    none, out = torch.empty(2, 0, 6 * 64, **bf16), torch.empty(2, 0, 6 * 64, **bf16)
    pool, table = torch.full((4, 2, 1, 16, 64), 3.0, **bf16), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    codes, ranges = torch.full((4, 2, 1, 16, 32), 5, dtype=torch.uint8, device="cuda"), torch.full((4, 2, 1, 16, 2), 2.0, **bf16)
    binding.rotary(none, out, 4, 1, turns)
    binding.paged_append(none, pool, table, 4, turns=turns, out=out)
    binding.paged_append4(none, codes, ranges, table, 4, turns=turns, out=out)
    binding.paged_load4(codes, ranges, table, torch.empty(2, 0, 2 * 64, **bf16))
    binding.status()
    assert (pool == 3).all() and (codes == 5).all() and (ranges == 2).all()
