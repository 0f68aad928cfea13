"""GPU: the gradient operators together, as a training step uses them, on W
replicas: look the tokens up, add the embedding's gradient to its place in each
replica's flat buffer (a bucket view), reduce, take the norm of the mean and
clip it, over two micro-batches (the first inside no_sync) and two steps.

Tolerance, set before the first run. u = 2^-24. Each element of a replica's
gradient is a sum of at most n fp32 terms (its tokens' rows in both
micro-batches, a few for the other parameters), then W terms are scaled and
folded, then one factor is applied: off by at most (n + 2 W + 10) u times the
sum of the terms' magnitudes, plus the factor's 6 u of the value (the norm's
own error among them: the norm of an error is at most the norm of its
bound)."""
import pytest

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.mark.parametrize("collective", [0, 1])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_a_training_step(collective, act):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bucketed_gradient_all_amd as ddp

    W, V, H, T, max_norm = 4, 500, 72, 900, 0.5
    numel = [V * H, 3000, 17]            # embedding, a weight, a bias
    plan = ddp.ddp_plan_buckets([4 * n for n in numel], ddp.DDP_ORDER_REVERSE, 40000, 8000)
    total = sum(numel)
    at, off = [0] * 3, 0
    for b, members in enumerate(plan.buckets()):
        for p in members:
            at[p] = off + int(plan.offset_in_bucket[p]) // 4
        off += int(plan.bucket_bytes[b]) // 4
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[act]
    code = {"f32": ddp.DDP_F32, "bf16": ddp.DDP_BF16}[act]
    scale = H ** 0.5
    scale32 = float(torch.tensor(scale, dtype=torch.float32))
    gen = torch.Generator().manual_seed(5)

    compute, comm = torch.cuda.Stream(), torch.cuda.Stream()
    flat = [torch.zeros(total, device="cuda") for _ in range(W)]
    table = torch.randn(V, H, generator=gen).to(dtype).cuda()
    torch.cuda.synchronize()
    r = ddp.make_reducer(W, numel, plan, ddp.DDP_IN_F32_VIEW, None, [f.data_ptr() for f in flat],
                         compute.cuda_stream, comm.cuda_stream, collective=collective)
    grads = ddp.make_reducer_grads(r)
    emb = ddp.EmbeddingDesc(V, H, table_dtype=code, grad_dtype=ddp.DDP_F32, act_dtype=code, scale=scale,
                            padding_idx=0)
    nbytes = ddp.ddp_embedding_grad_workspace_bytes(emb, T)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    norm = torch.zeros((), device="cuda")
    out = torch.empty(T, H, dtype=dtype, device="cuda")

    for step in range(2):
        mean = torch.zeros(total, dtype=torch.float64)
        size = torch.zeros(total, dtype=torch.float64)
        count = torch.zeros(total, dtype=torch.float64)
        for f in flat:
            f.zero_()
        torch.cuda.synchronize()
        for micro in range(2):
            ddp.ddp_set_require_sync(r, micro == 1)
            ddp.ddp_prepare_for_backward(r)
            for w in range(W):
                tok = (torch.rand(T, generator=gen) ** 3 * V).long()
                rows = torch.randn(T, H, generator=gen).to(dtype)
                other = torch.randn(3017, generator=gen)
                dtok, drows, dother = tok.cuda(), rows.cuda(), other.cuda()
                torch.cuda.synchronize()
                with torch.cuda.stream(compute):
                    ddp.ddp_embedding_lookup(emb, table.data_ptr(), dtok.data_ptr(), T, out.data_ptr(),
                                             compute.cuda_stream)
                    flat[w][at[1]:at[1] + 3000] += dother[:3000]
                    flat[w][at[2]:at[2] + 17] += dother[3000:]
                    ddp.ddp_embedding_grad(emb, drows.data_ptr(), dtok.data_ptr(), T, flat[w].data_ptr() + 4 * at[0],
                                           True, ws.data_ptr(), nbytes, compute.cuda_stream)
                torch.cuda.synchronize()
                want_out = table.cpu()[tok].double() * scale32
                u = torch.finfo(dtype).eps / 2
                assert bool(((out.cpu().double() - want_out).abs() <= want_out.abs() * (u + U32) * 1.001).all())
                keep = tok != 0
                e = torch.zeros(V, H, dtype=torch.float64).index_add_(0, tok[keep], rows.double()[keep] * scale32)
                m = torch.zeros(V, H, dtype=torch.float64).index_add_(0, tok[keep], rows.double()[keep].abs() * scale32)
                n = torch.bincount(tok[keep], minlength=V).double()
                mean[at[0]:at[0] + V * H] += e.reshape(-1) / W
                size[at[0]:at[0] + V * H] += m.reshape(-1) / W
                count[at[0]:at[0] + V * H] += n.repeat_interleave(H)
                for p, x in ((1, other[:3000]), (2, other[3000:])):
                    mean[at[p]:at[p] + numel[p]] += x.double() / W
                    size[at[p]:at[p] + numel[p]] += x.double().abs() / W
                    count[at[p]:at[p] + numel[p]] += 1
            ddp.ddp_mark_ready_many(r, [2, 1, 0])
            ddp.ddp_finish(r)
        ddp.ddp_clip_grad_norm(grads, ddp.DDP_NORM_L2, max_norm, norm.data_ptr(), compute.cuda_stream)
        torch.cuda.synchronize()
        bound = (count + 2 * W + 10) * U32 * size
        want = float(mean.norm())
        assert abs(float(norm) - want) <= float(bound.norm()) + 2 * U32 * want
        f = max_norm / (want + 1e-6)
        assert f < 1.0
        tol = f * (bound + mean.abs() * (float(bound.norm()) / want + 8 * U32))
        for b in range(plan.n_buckets):
            start = sum(int(x) for x in plan.bucket_bytes[:b]) // 4
            n = int(plan.bucket_bytes[b]) // 4
            q = -(-n // W)
            for w in range(W):
                lo, hi = (min(n, w * q), min(n, (w + 1) * q)) if collective else (0, n)
                part = slice(start + lo, start + hi)
                assert bool(((flat[w][part].cpu().double() - mean[part] * f).abs() <= tol[part]).all()), (step, b, w)
    ddp.ddp_grads_destroy(grads)
    ddp.ddp_reducer_destroy(r)
