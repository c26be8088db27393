"""The long-context operators called from several host threads at once, each with its own tensors and stream and with
sizes that want different amounts of shared memory: equal bit for bit to the same calls from one thread."""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from gpu_util import dev_bf16, dev_f32, dev_i32, rand_bf16  # noqa: E402


def _decode(B, rows):
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(B)
    H, D, page = 4, 64, 16
    table = np.zeros((B, rows // page), np.int32)
    table[:, :4] = np.arange(4 * B).reshape(B, 4)
    pool, table = dev_bf16(rand_bf16(rng, (4 * B, 2, 2, page, D))), dev_i32(table)
    lens, qkv = dev_i32(rng.integers(0, 60, B)), dev_bf16(rand_bf16(rng, (B, 8 * D)))

    def call(stream):
        y = torch.empty(B, H * D, dtype=torch.bfloat16, device="cuda")
        binding.paged_attention(qkv, pool, table, lens, y, H, stream=stream)
        return [y]
    return call


def _evict(rows, budget):
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(rows)
    page, Hkv = 16, 2
    n, more = rows // page, (budget + page - 1) // page
    pool, weight = dev_bf16(rand_bf16(rng, (n + more, 2, Hkv, page, 32))), dev_f32(rng.random((n + more, Hkv, page)))
    table, dst, lens = dev_i32(np.arange(n)[None]), dev_i32(n + np.arange(more)[None]), dev_i32([rows])

    def call(stream):
        new, kept = torch.empty_like(lens), torch.empty(1, Hkv, budget, dtype=torch.int32, device="cuda")
        binding.paged_evict(pool, weight, table, lens, dst, new, kept, budget, 2, 3, stream=stream)
        return [new, kept]
    return call


def test_threads_with_different_sizes(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    calls = [_decode(B, 8192) for B in (3, 700, 1500, 2500)] + [_evict(r, r // 3) for r in (480, 1600, 3200, 9600, 64000)]
    torch.cuda.synchronize()
    results, failed = [None] * len(calls), []
    start = threading.Barrier(len(calls))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                outs = [calls[i](stream) for _ in range(50)]
                stream.synchronize()
            assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(outs[0], o))
            results[i] = outs[0]
        except Exception as e:                                           # noqa: BLE001 (shown by the main thread)
            failed.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    binding.status()
    for call, r in zip(calls, results):
        want = call(torch.cuda.current_stream())
        assert all(torch.equal(a, b) for a, b in zip(want, r))
