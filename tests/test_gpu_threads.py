"""Calls from several threads at once, each on a stream of its own, the process's first calls among
them: the results are those of the same calls made one after another."""
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def jobs(seed):
    """Calls of every kind that share host-side state, on inputs of their own: () -> tensors."""
    from mla_latent_kv_16_gb300 import capi
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    out = []
    for heads, page, cache in ((128, 64, "bf16"), (128, 16, "e4m3"), (16, 8, "bf16"), (16, 5, "bf16"), (16, 8, "f32")):
        t = torch.float32 if cache == "f32" else torch.bfloat16
        batch, pages = 3, -(-300 // page)
        rows, scales = rnd(batch * pages, page, 576), None
        if cache == "e4m3":
            rows, scales = rows.to(torch.float8_e4m3fn).view(torch.uint8), rnd(batch * pages, page, 5).abs()
        else:
            rows = rows.to(t)
        table = torch.randperm(batch * pages, generator=g, device="cuda").int().view(batch, pages)
        lens = torch.tensor([300, 1, 299], dtype=torch.int32, device="cuda")
        q, qr = rnd(batch, 1, heads, 512).to(t), rnd(batch, 1, heads, 64).to(t)
        out.append(lambda a=(q, qr, rows, scales, table, lens, page, cache): capi.mla_decode_window(*a, 70, 5, num_splits=2))
        out.append(lambda a=(q, qr, rows, scales, table, lens, page, cache): capi.mla_decode_paged(*a, num_splits=3))
    w = [(rnd(4, 128, 512) / 512 ** 0.5).bfloat16() for _ in range(2)]
    q, qr, rows = rnd(150, 4, 128).bfloat16(), rnd(150, 4, 64).bfloat16(), rnd(200, 576).bfloat16()
    out.append(lambda: capi.mla_prefill_window(q, qr, rows, *w, 40, 3))
    out.append(lambda: capi.mla_prefill_mha(q, qr, rows, *w))
    out.append(lambda: (capi.mla_absorb_q(q, w[0]), capi.mla_linear(rows[:, :512].contiguous(), w[0].view(-1, 512))))
    table = torch.full((4, 8), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(40, dtype=torch.int32, device="cuda")
    seqs, grow = torch.arange(4, dtype=torch.int32, device="cuda"), torch.tensor([9, 0, 30, 1], dtype=torch.int32, device="cuda")

    def pages_call():
        t, n, r = table.clone(), lens.clone(), refs.clone()
        made = capi.mla_cache_extend(seqs, seqs, grow, t, n, r, 8, max_new=40)
        capi.mla_cache_free(seqs[:1], t, n, r, 8)
        return t, n, r, *made, *capi.mla_cache_compact(t, r)

    out.append(pages_call)
    return out


def main(threads=6):
    """The first calls of this process, from all threads at once; then the same ones in order."""
    got, errors = {}, []
    start = threading.Barrier(threads)
    work = [jobs(k) for k in range(threads)]
    torch.cuda.synchronize()

    def run(k):
        try:
            n = len(work[k])
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for turn in range(3):
                    for i in range(n):
                        j = (i + 2 * k) % n  # (each thread begins with another call)
                        got[k, j, turn] = [x for x in work[k][j]() if x is not None]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the parent)
            errors.append(repr(e))

    pool = [threading.Thread(target=run, args=(k,)) for k in range(threads)]
    [t.start() for t in pool]
    [t.join() for t in pool]
    assert not errors, errors
    torch.cuda.synchronize()
    for (k, j, turn), x in got.items():
        want = [y for y in work[k][j]() if y is not None]
        assert all(torch.equal(a, b) for a, b in zip(x, want)), (k, j, turn)
    print("threads ok")


def test_first_calls_from_many_threads():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from mla_latent_kv_16_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", "import test_gpu_threads as t; t.main()"], cwd=HERE, capture_output=True, text=True,
                       timeout=300, env={**os.environ, "PYTHONPATH": os.pathsep.join([os.path.dirname(HERE), HERE])})
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout + r.stderr
