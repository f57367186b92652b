"""A state-space layer as a model has it: the norm with the residual's addition, a projection,
the short convolution, the selective scan with its gate, a projection back.  Trained (gradients of
every weight) and served (prompts in chunks, then token by token, on pools of states)."""
import pytest
import torch

import chunked_gated_delta_rule_gb300 as gdr
from layer_ref import close, offsets, rms_norm, selective_scan, short_conv, wide

pytestmark = pytest.mark.gpu
WIDTH, C, S, TAPS = 48, 96, 16, 4


def weights(seed=0):
    gen = torch.Generator().manual_seed(seed)

    def randn(*shape, by=1.0):
        return (by * torch.randn(*shape, generator=gen)).cuda()

    return dict(norm=1.0 + randn(WIDTH, by=0.1), into=randn(WIDTH, 2 * C, by=WIDTH ** -0.5),
                taps=randn(C, TAPS, by=0.5), bias=randn(C, by=0.1), bc=randn(C, 2 * S, by=C ** -0.5),
                dt=randn(C, C, by=C ** -0.5), dt_bias=randn(C) - 2.0, A=-torch.exp(randn(C, S)),
                D=1.0 + randn(C, by=0.1), out=randn(C, WIDTH, by=C ** -0.5))


def trained(w, x, res, lens):
    cu = offsets(lens).cuda()
    h, r = gdr.rms_norm(x, w["norm"], res)
    xz = h @ w["into"]
    u, _ = gdr.short_conv(xz[..., :C], w["taps"], w["bias"], cu_seqlens=cu, max_seqlen=max(lens))
    bc = (u @ w["bc"]).reshape(1, -1, 2, 1, S)
    y, _ = gdr.selective_scan(u, u @ w["dt"], w["A"], bc[:, :, 0], bc[:, :, 1], w["D"], xz[..., C:],
                              w["dt_bias"], cu_seqlens=cu, max_seqlen=max(lens))
    return r + y @ w["out"]


def exact(w, x, res, lens):
    r = x + res
    xz = rms_norm(r, w["norm"], 1e-6)[0] @ w["into"]
    u, _ = short_conv(xz[:, :C], w["taps"], w["bias"], lens)
    bc = (u @ w["bc"]).reshape(-1, 2, 1, S)
    y, _ = selective_scan(u, u @ w["dt"], w["A"], bc[:, 0], bc[:, 1], w["D"], xz[:, C:], w["dt_bias"], lens)
    return r + (y @ w["out"])[None]


def test_trained():
    """FP32 against 64 bits: five operators of 1e-5 each, and products that carry what comes in on
    with factors of about one."""
    lens = [70, 1, 0, 130, 9]
    w = weights()
    gen = torch.Generator().manual_seed(1)
    x, res, dy = (torch.randn(1, sum(lens), WIDTH, generator=gen).cuda() for _ in range(3))
    leaf = {k: v.clone().requires_grad_() for k, v in dict(w, x=x, res=res).items()}
    y = trained(leaf, leaf["x"], leaf["res"], lens)
    (y * dy).sum().backward()
    ref = {k: wide(v) for k, v in dict(w, x=x, res=res).items()}
    want = exact(ref, ref["x"], ref["res"], lens)
    (want * dy.cpu().double()).sum().backward()
    close("y", y, want, work=1e-4)
    for k in leaf:
        close("d" + k, leaf[k].grad, ref[k].grad, work=1e-4)


class Server:
    """The layer on pools of states; a step takes new tokens of some of the sequences."""

    def __init__(self, w, rows):
        self.w = w
        self.conv = torch.zeros(rows, TAPS - 1, C, device="cuda")
        self.scan = torch.zeros(rows, C, S, device="cuda")

    def step(self, x, res, lens, rows):
        w, cu = self.w, offsets(lens).cuda()
        idx = torch.tensor(rows, dtype=torch.int32).cuda()
        h, r, _ = gdr.gdr_rms_norm_fwd(x, w["norm"], res)
        xz = h @ w["into"]
        u, _ = gdr.gdr_short_conv_fwd(xz[..., :C], w["taps"], w["bias"], cu, state=self.conv,
                                      state_indices=idx, max_seqlen=max(lens))
        bc = (u @ w["bc"]).reshape(1, -1, 2, 1, S)
        y, _ = gdr.gdr_selective_scan_fwd(u, u @ w["dt"], w["A"], bc[:, :, 0], bc[:, :, 1], w["D"],
                                          xz[..., C:], w["dt_bias"], cu, state=self.scan,
                                          state_indices=idx, max_seqlen=max(lens))
        return r + y @ w["out"]


def test_served():
    """Three sequences, their prompts in chunks of up to 40 tokens and then token by token, one of
    them joining late; against all their tokens in 64 bits."""
    total, prompts, rows = [97, 60, 130], [90, 50, 121], [4, 0, 2]
    w = weights()
    gen = torch.Generator().manual_seed(2)
    x, res = (torch.randn(1, sum(total), WIDTH, generator=gen).cuda() for _ in range(2))
    first = [0, total[0], total[0] + total[1]]
    server, at, got = Server(w, 6), [0, 0, 0], [[], [], []]
    for step in range(100):
        who = [i for i in range(3) if at[i] < total[i] and (i != 1 or step >= 2)]
        if not who:
            break
        lens = [min(40, prompts[i] - at[i]) if at[i] < prompts[i] else 1 for i in who]
        part = [torch.cat([t[:, first[i] + at[i]:first[i] + at[i] + n] for i, n in zip(who, lens)], 1)
                for t in (x, res)]
        y = server.step(*part, lens, [rows[i] for i in who])
        for i, n, piece in zip(who, lens, y.split(lens, 1)):
            got[i].append(piece)
            at[i] += n
    assert at == total
    want = exact({k: v.cpu().double() for k, v in w.items()}, x.cpu().double(), res.cpu().double(), total)
    close("y", torch.cat([torch.cat(g, 1) for g in got], 1), want, work=1e-4)
    assert not server.conv[[1, 3, 5]].any() and not server.scan[[1, 3, 5]].any()


def test_decode_step_in_a_graph():
    """A captured decode step, replayed: the states move on with every replay, as they do with
    eager calls."""
    w, n = weights(), 3
    gen = torch.Generator().manual_seed(3)
    x, res = (torch.randn(1, n, WIDTH, generator=gen).cuda() for _ in range(2))
    idx = torch.tensor([2, 0, 1], dtype=torch.int32).cuda()
    cu = offsets([1] * n).cuda()

    def step(conv, scan):
        h, r, _ = gdr.gdr_rms_norm_fwd(x, w["norm"], res)
        xz = h @ w["into"]
        u, _ = gdr.gdr_short_conv_fwd(xz[..., :C], w["taps"], w["bias"], cu, state=conv,
                                      state_indices=idx, max_seqlen=1)
        bc = (u @ w["bc"]).reshape(1, -1, 2, 1, S)
        y, _ = gdr.gdr_selective_scan_fwd(u, u @ w["dt"], w["A"], bc[:, :, 0], bc[:, :, 1], w["D"],
                                          xz[..., C:], w["dt_bias"], cu, state=scan,
                                          state_indices=idx, max_seqlen=1)
        return r + y @ w["out"]

    pools = [(torch.zeros(n, TAPS - 1, C, device="cuda"), torch.zeros(n, C, S, device="cuda"))
             for _ in range(2)]
    step(*(p.clone() for p in pools[0]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(*pools[0])
    for p in pools[0]:
        p.zero_()
    for i in range(4):
        x.copy_(torch.randn(1, n, WIDTH, generator=gen))
        graph.replay()
        assert torch.equal(y, step(*pools[1])), i
    for a, b in zip(*pools):
        assert torch.equal(a, b)


def test_another_stream():
    """Calls on a side stream on tensors made on the current one: the same bits, and memory that
    is let go at once is not handed out under them."""
    lens = [300, 200]
    w = weights()
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(1, 500, C, generator=gen).cuda()
    bc = torch.randn(1, 500, 2, 1, S, generator=gen).cuda()
    cu = offsets(lens).cuda()
    args = (x, x, w["A"], bc[:, :, 0], bc[:, :, 1])
    want, ht = gdr.gdr_selective_scan_fwd(*args, cu_seqlens=cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        got = gdr.gdr_selective_scan_fwd(*args, cu_seqlens=cu, stream=side)
        del got
        torch.empty(500 * C, device="cuda").fill_(float("nan"))
        outs.append(gdr.gdr_selective_scan_fwd(*args, cu_seqlens=cu, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    for y, h in outs:
        assert torch.equal(y, want) and torch.equal(h, ht)
