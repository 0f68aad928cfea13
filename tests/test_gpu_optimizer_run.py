"""GPU: the operators around the reduction together, as a training step uses
them: embedding lookup, layer norm with its residual, both backward passes
straight into the replicas' flat buffers, the reduction, the norm of its results,
and the AdamW step clipped by it. Checked against the gradients in 64 bits,
between the all-reduce and the reduce-scatter (bit for bit), and replayed from a
graph (bit for bit).

The first step from zero moments moves a parameter by lr * g / (|g| + eps) and
the decay. Where |g| is at least 1e-3 of its tensor's largest and at least 1e-6,
100 times eps, its relative error d changes that by at most lr * d * eps / |g|,
1e-2 d lr. The chain's error is at most 1000 u of a tensor's largest gradient (sums
of a few hundred terms), so d is at most 1e6 u = 0.06, and the step is off by
1e-3 lr at most, besides 4 u of the parameter.
"""
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
W, T, V, H = 2, 300, 97, 260
LR, EPS, DECAY, MAX_NORM = 1e-3, 1e-8, 0.1, 0.5


class Run:
    """Two replicas of an embedding and a layer norm; the loss is the sum of
    the output times fixed random numbers."""

    def __init__(self, collective, bits):
        import torch
        import bucketed_gradient_all_amd as ddp
        self.ddp, self.torch, self.collective, self.bits = ddp, torch, collective, bits
        g = torch.Generator().manual_seed(3)
        rand = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
        self.tokens = [torch.randint(0, V, (T,), generator=g).cuda() for _ in range(W)]
        self.pos, self.dy = rand(T, H), [rand(T, H) * 0.1 for _ in range(W)]
        numel = [V * H, H, H]                       # table, weight, bias
        plan = ddp.ddp_plan_buckets([4 * n for n in numel], cap_bytes=4096, first_cap_bytes=1024)
        at, self.where = 0, [0] * 3                 # element offsets in the flat buffer
        for k, members in enumerate(plan.buckets()):
            for p in members:
                self.where[p] = at // 4 + int(plan.offset_in_bucket[p]) // 4
            at += int(plan.bucket_bytes[k])
        self.numel, n = numel, at // 4
        start = torch.cat([rand(V * H) * 0.5, 1.0 + 0.1 * rand(H), 0.1 * rand(H)])
        self.params, self.flat = [], []
        for _ in range(W):
            p = torch.empty(n, device="cuda")
            for i, (o, k) in enumerate(zip(self.where, numel)):
                p[o:o + k] = start[sum(numel[:i]):sum(numel[:i]) + k]
            self.params.append(p)
            self.flat.append(torch.zeros(n, device="cuda"))
        self.start = self.params[0].clone()
        s = torch.cuda.current_stream().cuda_stream
        self.comm = torch.cuda.Stream()
        self.reducer = ddp.make_reducer(W, numel, plan, ddp.DDP_IN_F32_VIEW, None, [f.data_ptr() for f in self.flat],
                                        s, self.comm.cuda_stream, collective=collective)
        self.grads = ddp.make_reducer_grads(self.reducer)
        # what each replica steps: everything after an all-reduce, its chunks after a reduce-scatter
        tensors = []
        for w in range(W):
            if collective == ddp.DDP_ALL_REDUCE:
                tensors += [(w, o, k, DECAY if i == 0 else 0.0) for i, (o, k) in enumerate(zip(self.where, numel))]
            else:
                at = 0
                for b, size in enumerate(plan.bucket_bytes):
                    k = int(size) // 4
                    q = -(-k // W)
                    lo, hi = min(k, w * q), min(k, (w + 1) * q)
                    for i, (o, m) in enumerate(zip(self.where, numel)):   # a chunk's part of each parameter
                        a, z = max(at + lo, o), min(at + hi, o + m)
                        if a < z:
                            tensors.append((w, a, z - a, DECAY if i == 0 else 0.0))
                    at += k
        self.tensors = tensors
        dtype = torch.float32 if bits == 32 else torch.uint8
        self.m, self.v = ([torch.zeros(k, dtype=dtype, device="cuda") for _, _, k, _ in tensors] for _ in range(2))
        self.ms, self.vs = ([torch.zeros(-(-k // 128), device="cuda") for _, _, k, _ in tensors] for _ in range(2))
        ptr = lambda ts: [t.data_ptr() for t in ts]   # noqa: E731
        self.opt = ddp.make_adamw(
            [k for _, _, k, _ in tensors], [self.flat[w].data_ptr() + 4 * o for w, o, _, _ in tensors],
            [self.params[w].data_ptr() + 4 * o for w, o, _, _ in tensors], ptr(self.m), ptr(self.v),
            state=ddp.DDP_STATE_F32 if bits == 32 else ddp.DDP_STATE_8BIT,
            m_scale_ptrs=ptr(self.ms) if bits == 8 else None, v_scale_ptrs=ptr(self.vs) if bits == 8 else None,
            weight_decay=[d for _, _, _, d in tensors])
        self.x, self.z, self.y, self.dx = ([torch.empty(T, H, device="cuda") for _ in range(W)] for _ in range(4))
        self.mean, self.rstd = ([torch.empty(T, device="cuda") for _ in range(W)] for _ in range(2))
        self.norm = torch.zeros(1, device="cuda")
        self.emb, self.ln = ddp.EmbeddingDesc(V, H, scale=2.0), ddp.LayerNormDesc(H)
        self.work = [torch.empty(max(ddp.ddp_embedding_grad_workspace_bytes(self.emb, T),
                                     ddp.ddp_layernorm_grad_workspace_bytes(self.ln, T)), dtype=torch.uint8,
                                 device="cuda") for _ in range(W)]

    def step(self, **at):
        """One step on the current stream; `at`: step, or step_ptr."""
        ddp, torch = self.ddp, self.torch
        s = torch.cuda.current_stream().cuda_stream
        ddp.ddp_prepare_for_backward(self.reducer)
        for w in range(W):
            self.flat[w].zero_()
            table, weight, bias = (self.params[w].data_ptr() + 4 * o for o in self.where)
            dtable, dweight, dbias = (self.flat[w].data_ptr() + 4 * o for o in self.where)
            ddp.ddp_embedding_lookup(self.emb, table, self.tokens[w].data_ptr(), T, self.x[w].data_ptr(), s)
            ddp.ddp_layernorm(self.ln, T, self.x[w].data_ptr(), weight, bias, self.y[w].data_ptr(), s,
                              add=self.pos.data_ptr(), z=self.z[w].data_ptr(), mean=self.mean[w].data_ptr(),
                              rstd=self.rstd[w].data_ptr())
            ws = self.work[w].data_ptr(), self.work[w].numel()
            ddp.ddp_layernorm_grad(self.ln, T, self.dy[w].data_ptr(), self.z[w].data_ptr(), weight,
                                   self.mean[w].data_ptr(), self.rstd[w].data_ptr(), self.dx[w].data_ptr(), dweight,
                                   dbias, True, *ws, s)
            ddp.ddp_embedding_grad(self.emb, self.dx[w].data_ptr(), self.tokens[w].data_ptr(), T, dtable, True, *ws, s)
        ddp.ddp_mark_ready_many(self.reducer, [2, 1, 0])
        ddp.ddp_finish(self.reducer)
        ddp.ddp_grad_norm(self.grads, ddp.DDP_NORM_L2, self.norm.data_ptr(), s)
        ddp.ddp_adamw_step(self.opt, LR, at.get("step", 0), s, eps=EPS, max_norm=MAX_NORM, norm=self.norm.data_ptr(),
                           skip_nonfinite=True, step_ptr=at.get("step_ptr", 0))
        if self.collective == ddp.DDP_REDUCE_SCATTER:   # the owners' shards to everyone
            for w, o, k, _ in self.tensors:
                for u in range(W):
                    if u != w:
                        self.params[u][o:o + k].copy_(self.params[w][o:o + k])

    def gradients64(self):
        torch = self.torch
        p = [self.start[o:o + k].double().requires_grad_() for o, k in zip(self.where, self.numel)]
        loss = 0.0
        for w in range(W):
            z = 2.0 * p[0].view(V, H)[self.tokens[w]] + self.pos.double()
            d = z - z.mean(1, keepdim=True)
            y = d * (d.square().mean(1, keepdim=True) + 1e-5).rsqrt() * p[1] + p[2]
            loss = loss + (y * self.dy[w].double()).sum() / W
        loss.backward()
        return [t.grad for t in p]

    def state(self):
        return [t.clone() for t in self.params + self.flat + self.m + self.v + self.ms + self.vs + [self.norm]]


def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("collective", [0, 1])
def test_first_step_against_the_gradients_in_64_bits(collective, bits):
    torch = _gpu()
    r = Run(collective, bits)
    want = r.gradients64()
    r.step(step=1)
    torch.cuda.synchronize()
    norm = torch.cat(want).norm()
    assert abs(float(r.norm) / float(norm) - 1) < 1000 * U
    f = min(1.0, MAX_NORM / (float(norm) + 1e-6))
    assert f < 1.0
    assert torch.equal(r.params[0], r.params[1])
    for i, (g, o, k) in enumerate(zip(want, r.where, r.numel)):
        g = g * f
        sure = (g.abs() >= 1e-3 * g.abs().max()) & (g.abs() >= 1e-6)
        assert sure.double().mean() > 0.5
        p0, p = r.start[o:o + k].double(), r.params[0][o:o + k].double()
        expected = p0 * (1.0 - LR * (DECAY if i == 0 else 0.0)) - LR * g / (g.abs() + EPS)
        off = (p - expected).abs()[sure] - 4 * U * p0.abs()[sure]
        assert off.max() <= 1e-3 * LR, (i, float(off.max()))


def test_a_sharded_run_equals_the_replicated_one():
    """Three steps: the owners' shards are the all-reduce's results, so are the
    parameters. The norm is summed over other tensors, in another order, in 64
    bits and rounded once: nearly always the same fp32 value, as here."""
    torch = _gpu()
    a, b = Run(0, 32), Run(1, 32)
    for k in (1, 2, 3):
        a.step(step=k)
        b.step(step=k)
        torch.cuda.synchronize()
        assert torch.equal(a.norm, b.norm)
        assert torch.equal(a.params[0], b.params[0]) and torch.equal(b.params[0], b.params[1]), k


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("collective", [0, 1])
def test_replayed_steps_equal_eager_ones(collective, bits):
    torch = _gpu()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a, b = Run(collective, bits), Run(collective, bits)
        count = torch.zeros(1, dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            count.add_(1)
            a.step(step_ptr=count.data_ptr())
        for k in range(1, 5):
            graph.replay()
            b.step(step=k)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(a.state(), b.state())), k
            for r in (a, b):   # other data for the next step
                for w in range(W):
                    r.tokens[w].add_(k).remainder_(V)
                    r.dy[w].mul_(1.5)
