"""DP-SGD with randomized clipping around the per-sample norm path.

The step follows 'Efficient DP-SGD for LLMs with Randomized Clipping'
(papernotes.org note, 方法详解 › 整体框架 and 损失函数 / 训练策略): one
forward pass in which a hook on every linear-like module records its input
activations A [B][T][d]; a first backward pass that yields each module's
output gradients G [B][T][p]; per module a norm estimate n_hat_i (Hutchinson
by default, Hutch++ or the exact norm on request) summed over the modules into
n_i; clip factors c_i = min(C / sqrt(n_i), 1); a second backward pass of the
rewritten loss sum_i c_i l_i, which gives sum_i c_i grad l_i; Gaussian noise
sigma C N(0, I) added to that sum; and the optimizer step.

Readings where the pages leave a step open:
  * The first backward pass is of sum_i l_i, so G_i is the gradient of sample
    i's own loss.
  * The noisy sum is divided by the batch size B before the optimizer, as in
    textbook DP-SGD; the pages add the noise to the aggregated gradient and
    do not state the averaging.
  * A weight applied several times in one forward pass (by one module called
    more than once, or by several linear modules that hold the same weight)
    has one per-sample gradient sum_u A_u^T G_u = [A_1; A_2; ...]^T
    [G_1; G_2; ...]: its recordings are concatenated along T.
  * A fresh projection P ~ N(0, 1/k) is drawn per weight and step.
  * The projections and the noise are internal randomness of the mechanism:
    by default each comes from its own generator seeded from the operating
    system's entropy, so neither can be replayed from the code. Fixed seeds
    exist for tests only.

Every norm estimate runs in libdpnorm on the GPU; torch runs the model and its
two backward passes. The weights that are clipped are those of bias-free
nn.Linear modules (Llama has no biases) and of layers.Embedding tables, whose
per-sample norm is exact whatever the estimator is: row v of sample i's
gradient is the sum of its output gradients at the positions of id v, so the
norm costs one pass over the output gradients. Refused, since part of a gradient would go unclipped: any other
trainable parameter, and a weight that a module of another kind also
holds (a tied embedding). A use of a weight that the hooks cannot see (the
weight passed to F.linear outside its module) is caught on the first step:
the clipped gradient autograd accumulates must equal sum_i c_i G_i^T A_i
from the recordings.

Every row of a recording has to belong to one sample, samples in order: a
module applied once to rows that all samples use (a learned position table
looked up as pos(arange(T)) and added to every sample) has output gradients
that are already summed over the samples, from which no norm of a sample can
be had. Ids whose first dimension is not the batch are refused, and the first
step's check finds what the shapes do not show: its first backward pass is of
sum_i w_i l_i with powers of two w_i in random order, and G_i is what it gives
divided by w_i, the same bits where a row is sample i's alone and something
else where it is not.
"""
from __future__ import annotations

import secrets
from typing import Callable, Dict, List, Optional, Tuple

import torch
from torch import nn

import sample_grad_norms_amd as dp
from sample_grad_norms_amd.layers import Embedding

ProjectionFn = Callable[[int, int, torch.dtype, torch.device, torch.Generator], torch.Tensor]


def gaussian_projection(p: int, k: int, dtype: torch.dtype, device: torch.device,
                        generator: torch.Generator) -> torch.Tensor:
    """P [p][k] with i.i.d. N(0, 1/k) entries, drawn in float32 and rounded
    once to `dtype`."""
    P = torch.randn(p, k, generator=generator, device=device, dtype=torch.float32) / (k ** 0.5)
    return P.to(dtype)


class RandomizedClipping:
    """Hooks a model's bias-free linear layers and embedding tables
    (layers.Embedding) and runs the DP-SGD-RC step.

    Usage::

        rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.8)
        with rc.capture():
            losses = per_sample_losses(model(x), y)      # float32 [B]
        n, c = rc.clip_factors(losses)                   # backward 1 + norms
        rc.clipped_backward(losses, c)                   # backward 2
        rc.add_noise()                                   # sigma C N(0, I), / B
        optimizer.step(); optimizer.zero_grad()

    or ``rc.step(losses, optimizer)`` for the last four lines.

    estimator: "hutch" (k Gaussian columns), "hutch_sign" (k +-1 columns stored
    as bits), "hutchpp" (budget k) or "exact".
    norm_dtype: element type handed to the norm path (bfloat16 or float32;
    default: the activations' own). Widths must suit that type (multiples of
    8 for bfloat16, 4 for float32).
    keep_layers: keep the (A, G, P) triples of the last step in
    ``last_layers`` (P is the sign words for "hutch_sign", the pair (S, P)
    of sketch and tail projection for "hutchpp", None for "exact").
    timer: an optional sample_grad_norms_amd.KernelTimer given to the grouped
    Hutchinson calls (per-launch times of the norm path).
    seed, noise_seed: FOR TESTS ONLY. Fixed seeds of the projection and noise
    generators make the mechanism's randomness reproducible by anyone who
    knows them, which voids its privacy; the default (None) seeds each from
    the operating system's entropy.
    verify_coverage: on the first step, check that each clipped weight's
    gradient from the second backward pass equals sum_i c_i G_i^T A_i from
    the recordings (it does not when the weight has a use the hooks cannot
    see, such as F.linear called with it outside its module, or when rows of
    a recording are not one sample's); a mismatch raises RuntimeError. The
    check assumes nothing else adds to the weights' .grad during that backward
    pass.

    Embedding ids are [B, ...]: one row of ids for each sample. Ids [B], one a
    sample, look like the positions of B samples of length B, which only the
    check can tell apart; without it they are refused ([B][1] is not).
    """

    def __init__(self, model: nn.Module, C: float, noise_multiplier: float, k: int = 32,
                 estimator: str = "hutch", norm_dtype: Optional[torch.dtype] = None, seed: Optional[int] = None,
                 projection: ProjectionFn = gaussian_projection, keep_layers: bool = False,
                 timer: Optional["dp.KernelTimer"] = None, noise_seed: Optional[int] = None,
                 verify_coverage: bool = True):
        if estimator not in ("hutch", "hutch_sign", "hutchpp", "exact"):
            raise ValueError("estimator must be 'hutch', 'hutch_sign', 'hutchpp' or 'exact'")
        if not C > 0:
            raise ValueError("C must be positive")
        self.C, self.sigma, self.k = float(C), float(noise_multiplier), int(k)
        self.estimator, self.norm_dtype, self.projection = estimator, norm_dtype, projection
        self.seed = seed if seed is not None else secrets.randbits(63)
        self.noise_seed = noise_seed if noise_seed is not None else secrets.randbits(63)
        self.keep_layers, self.timer = keep_layers, timer
        self.last_layers: List[Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]] = []
        self.modules: List[nn.Linear] = [m for m in model.modules() if isinstance(m, nn.Linear)]
        for m in self.modules:
            if m.bias is not None:
                raise ValueError("linear layers with a bias are not supported (the clipped gradient would miss it)")
        self.tables: List[Embedding] = [m for m in model.modules() if isinstance(m, Embedding)]
        covered = {id(m.weight) for m in self.modules}
        # a weight that a module of another kind also holds (a tied
        # embedding) gets gradient through that module, which no hook sees
        tied = [f"{name}.{pname}" if name else pname for name, mod in model.named_modules()
                if not isinstance(mod, nn.Linear)
                for pname, p in mod.named_parameters(recurse=False) if id(p) in covered]
        if tied:
            raise ValueError(f"linear weights shared with modules that are not linear layers would go partly "
                             f"unclipped: {tied}")
        covered_tables = {id(m.weight) for m in self.tables}
        shared = [f"{name}.{pname}" if name else pname for name, mod in model.named_modules()
                  if not isinstance(mod, Embedding)
                  for pname, p in mod.named_parameters(recurse=False) if id(p) in covered_tables]
        if shared:
            raise ValueError(f"embedding tables shared with modules that are not layers.Embedding would go partly "
                             f"unclipped: {shared}")
        covered |= covered_tables
        loose = [name for name, p in model.named_parameters(remove_duplicate=False)
                 if p.requires_grad and id(p) not in covered]
        if loose:
            raise ValueError(f"trainable parameters outside bias-free linear layers would go unclipped: {loose}")
        # one entry per distinct weight, in module order (modules holding the
        # same weight contribute to one per-sample gradient)
        self.params: List[nn.Parameter] = []
        self._users: Dict[int, List[nn.Linear]] = {}
        for m in self.modules:
            if id(m.weight) not in self._users:
                self._users[id(m.weight)] = []
                if m.weight.requires_grad:
                    self.params.append(m.weight)
            self._users[id(m.weight)].append(m)
        for t in self.tables:
            if t.weight.requires_grad and all(p is not t.weight for p in self.params):
                self.params.append(t.weight)
        self._names = {id(p): name for name, p in model.named_parameters()}
        self._capturing = False
        self._rec: Dict[nn.Module, List[Tuple[torch.Tensor, torch.Tensor]]] = {}
        self._gen: Optional[torch.Generator] = None
        self._noise_gen: Optional[torch.Generator] = None
        self._batch = 0
        self._verify = bool(verify_coverage)   # on the next step
        self._verified = False
        self._pending: Optional[List[Tuple[nn.Parameter, torch.Tensor, torch.Tensor]]] = None
        # per table of the last step: (weight, order of its ids, output gradients, scale)
        self._table_recs: List[Tuple[nn.Parameter, dp.EmbedOrder, torch.Tensor, float]] = []
        self._handles = [m.register_forward_hook(self._hook) for m in [*self.modules, *self.tables]]

    # -- capture ---------------------------------------------------------
    def _hook(self, module, inputs, output):
        if self._capturing and module.weight.requires_grad:
            self._rec.setdefault(module, []).append((inputs[0], output))

    class _Capture:
        def __init__(self, rc):
            self.rc = rc

        def __enter__(self):
            self.rc._rec = {}
            self.rc._capturing = True
            return self.rc

        def __exit__(self, *exc):
            self.rc._capturing = False
            return False

    def capture(self):
        """Context in which the model's forward pass is recorded."""
        return RandomizedClipping._Capture(self)

    def remove(self):
        for h in self._handles:
            h.remove()
        self._handles = []

    # -- the step --------------------------------------------------------
    def _generator(self, device):
        if self._gen is None:
            self._gen = torch.Generator(device=device)
            self._gen.manual_seed(self.seed)
        return self._gen

    def _noise_generator(self, device):
        if self._noise_gen is None:
            self._noise_gen = torch.Generator(device=device)
            self._noise_gen.manual_seed(self.noise_seed)
        return self._noise_gen

    def _collect(self, losses: torch.Tensor) -> List[Tuple[torch.Tensor, torch.Tensor]]:
        """Backward pass 1: per recorded weight, (A [B][T'][d], G [B][T'][p])
        with every use of the weight concatenated along T."""
        if losses.dim() != 1:
            raise ValueError("losses must be the per-sample losses [B]")
        if not self._rec:
            raise RuntimeError("no forward pass was captured (run the model inside rc.capture())")
        B = losses.shape[0]
        for m in self.tables:
            for tok, _ in self._rec.get(m, []):
                self._check_ids(m, tok, B)
        weights = []   # (weight, [(input, output), ...]) in module order
        for m in self.modules:
            if m in self._rec:
                key = id(m.weight)
                if not weights or all(id(w) != key for w, _ in weights):
                    weights.append((m.weight, [r for u in self._users[key] for r in self._rec.get(u, [])]))
        outputs = [o for _, recs in weights for (_, o) in recs]
        # the uses of every table, by the scale of the look-up
        looked = {}
        for m in self.tables:
            for r in self._rec.get(m, []):
                looked.setdefault((id(m.weight), m.scale), (m, []))[1].append(r)
        outputs += [o for _, recs in looked.values() for (_, o) in recs]
        # the step that is checked: powers of two, whose product and quotient are exact
        w, unweighted = None, None
        if self._verify and B > 1 and all(o.dtype in (torch.bfloat16, torch.float32, torch.float64) for o in outputs):
            w = self._sample_weights(B, losses.device)
            unweighted = (1.0 / w).view(B, 1, 1)
        total = losses.sum() if w is None else (w.to(losses.dtype) * losses).sum()
        grads = torch.autograd.grad(total, outputs, retain_graph=True, allow_unused=True)

        def by_sample(g):
            g = g.detach().reshape(B, -1, g.shape[-1])
            return g if unweighted is None else g * unweighted.to(g.dtype)

        layers, at, cast = [], 0, {}
        for w, recs in weights:
            As, Gs = [], []
            for (a, out), g in zip(recs, grads[at:at + len(recs)]):
                if g is None:  # the output did not reach the loss
                    g = torch.zeros_like(out)
                As.append(self._cast(a.detach().reshape(B, -1, a.shape[-1]), cast))
                Gs.append(self._cast(by_sample(g), cast))
            at += len(recs)
            A = As[0] if len(As) == 1 else torch.cat(As, dim=1)
            G = Gs[0] if len(Gs) == 1 else torch.cat(Gs, dim=1)
            layers.append((A, G))
        scales = [w for w, _ in looked]
        split = [w for w in scales if scales.count(w) > 1]
        if split:
            raise ValueError("one embedding table looked up with two scales has no norm of its own: use one scale")
        self._table_recs = []
        for m, recs in looked.values():
            toks, Gs = [], []
            for (tok, out), g in zip(recs, grads[at:at + len(recs)]):
                if g is None:
                    g = torch.zeros_like(out)
                toks.append(tok.detach().reshape(B, -1))
                Gs.append(self._cast(by_sample(g), cast))
            at += len(recs)
            tok = toks[0] if len(toks) == 1 else torch.cat([t.long() for t in toks], dim=1)
            G = Gs[0] if len(Gs) == 1 else torch.cat(Gs, dim=1)
            self._table_recs.append((m.weight, dp.embed_order(tok.contiguous(), m.weight.shape[0]), G, m.scale))
        self._pending = [(w, A, G) for (w, _), (A, G) in zip(weights, layers)] if self._verify else None
        self._batch = B
        self._rec = {}
        return layers

    def _check_ids(self, table: Embedding, tok: torch.Tensor, B: int) -> None:
        """The ids of a look-up are [B, ...], so that every row of its output is one sample's."""
        name = self._names.get(id(table.weight), "")
        if tok.dim() == 0 or tok.shape[0] != B:
            raise ValueError(f"table {name} is looked up with ids {list(tok.shape)}: they must be [B={B}, ...], a row for "
                             f"each sample (a position table: arange(T).expand(B, T))")
        if tok.dim() == 1 and B > 1 and not (self._verify or self._verified):
            raise ValueError(f"table {name} is looked up with ids [B={B}], which may as well be positions that all samples "
                             f"share: give one id a sample as [B][1], or leave verify_coverage on")

    @staticmethod
    def _sample_weights(B: int, device: torch.device) -> torch.Tensor:
        """Powers of two in random order, each of eight before one comes again
        (and no draw from the generators that a program seeds)."""
        rng = secrets.SystemRandom()
        return torch.tensor([2.0 ** e for _ in range(0, B, 8) for e in rng.sample(range(8), 8)][:B], device=device)

    def clip_factors(self, losses: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """Backward pass 1 and the norm path: returns (n, c), float32 [B]."""
        layers = self._collect(losses)
        B = losses.shape[0]
        device = layers[0][0].device if layers else self._table_recs[0][2].device
        gen = self._generator(device)
        n = torch.zeros(B, dtype=torch.float32, device=device)
        used = []
        if self.estimator in ("hutch", "hutch_sign"):
            if self.estimator == "hutch":
                triples = [(A, G, self.projection(G.shape[2], self.k, A.dtype, device, gen)) for (A, G) in layers]
            else:
                triples = [(A, G, dp.random_signs(G.shape[2], self.k, device=device, generator=gen))
                           for (A, G) in layers]
            # one grouped call per sequence length (a module applied u times has u T rows)
            lengths = sorted({A.shape[1] for (A, _, _) in triples})
            for j, T in enumerate(lengths):
                part = [t for t in triples if t[0].shape[1] == T]
                if self.estimator == "hutch":
                    dp.hutch_grouped(part, out=n, accumulate=j > 0, timer=self.timer)
                else:
                    dp.hutch_sign_grouped(part, self.k, out=n, accumulate=j > 0)
            used = triples
        else:
            for (A, G) in layers:
                if self.estimator == "exact":
                    dp.exact(A, G, out=n, accumulate=True)
                    used.append((A, G, None))
                else:
                    m_s, m_t = dp.hutchpp_split(self.k)
                    S = torch.randn(G.shape[2], m_s, generator=gen, device=device).to(A.dtype)
                    P = self.projection(G.shape[2], m_t, A.dtype, device, gen)
                    dp.hutchpp(A, G, S, P, k=self.k, out=n, accumulate=True)
                    used.append((A, G, (S, P)))
        for (_, order, G, scale) in self._table_recs:
            dp.embed_norm(order, G, scale=scale, out=n, accumulate=True)
        if self._pending is None:   # (no check will read them)
            self._table_recs = []
        c = dp.clip_factors(n, self.C)
        self.last_layers = used if self.keep_layers else []
        return n, c

    def _cast(self, t: torch.Tensor, cache: dict) -> torch.Tensor:
        # layers reading one tensor keep sharing one copy (and one pass over it); the
        # tensor stays with its copy, so that no other can come to lie at its address
        dt = self.norm_dtype or t.dtype
        key = (t.data_ptr(), tuple(t.shape), t.stride(), t.dtype)
        if key not in cache:
            cache[key] = (t.to(dt).contiguous(), t)
        return cache[key][0]

    def clipped_backward(self, losses: torch.Tensor, c: torch.Tensor) -> None:
        """Backward pass 2: accumulates sum_i c_i grad l_i into the weights' .grad
        (on the first step, then checked against the recordings)."""
        pending, self._pending = self._pending, None
        tables, self._table_recs = self._table_recs, []
        before = None
        if pending is not None:
            before = [w.grad.detach().float().clone() if w.grad is not None else None
                      for w in [w for w, _, _ in pending] + [w for w, _, _, _ in tables]]
        (c.detach().to(losses.dtype) * losses).sum().backward()
        if pending is not None:
            self._check_coverage(pending, before, c)
            cw = c.detach().float()
            for (w, order, G, scale), g0 in zip(tables, before[len(pending):]):
                want = dp.embed_grad(order, G, scale=scale, weights=cw).float()
                self._check_gradient(w, want, g0)
            self._verify, self._verified = False, True

    def _check_coverage(self, pending, before, c: torch.Tensor) -> None:
        """Each weight's gradient from backward pass 2 must be sum_i c_i G_i^T A_i
        over its recordings (within the rounding of the recorded dtype)."""
        cw = c.detach().float()
        for (w, A, G), g0 in zip(pending, before):
            if not w.requires_grad:
                continue
            B, T, d = A.shape
            p = G.shape[2]
            self._check_gradient(w, (G.float() * cw.view(B, 1, 1)).reshape(B * T, p).t() @ A.float().reshape(B * T, d), g0)

    def _check_gradient(self, w: nn.Parameter, want: torch.Tensor, g0: Optional[torch.Tensor]) -> None:
        """The weight's gradient less what it held before (g0) against `want`."""
        got = torch.zeros_like(want) if w.grad is None else w.grad.detach().float()
        if g0 is not None:
            got = got - g0
        scale = float(torch.linalg.vector_norm(want))
        err = float(torch.linalg.vector_norm(got - want))
        if err > 5e-2 * scale + 1e-30:
            raise RuntimeError(
                f"the gradient of weight {self._names.get(id(w), '')} {list(w.shape)} differs from what its "
                f"recorded uses give (relative {err / max(scale, 1e-300):.2e}): it has a use the hooks do not "
                f"see (e.g. F.linear called with it outside its module), which would go unclipped, or rows of a "
                f"recording are not one sample's (e.g. a layer applied once to rows that all samples use)")

    def add_noise(self) -> None:
        """Adds sigma C N(0, I) to each clipped gradient sum and divides by B."""
        if self._batch <= 0:
            raise RuntimeError("clip_factors has not run for this step")
        for p in self.params:
            if p.grad is None:
                p.grad = torch.zeros_like(p)
            g = p.grad.float()
            if self.sigma > 0:
                g = g + self.sigma * self.C * torch.randn(p.shape, generator=self._noise_generator(p.device),
                                                          device=p.device, dtype=torch.float32)
            p.grad.copy_((g / self._batch).to(p.grad.dtype))
        self._batch = 0

    def step(self, losses: torch.Tensor, optimizer: torch.optim.Optimizer) -> Tuple[torch.Tensor, torch.Tensor]:
        """clip_factors, clipped_backward, add_noise, optimizer.step, zero_grad."""
        n, c = self.clip_factors(losses)
        self.clipped_backward(losses, c)
        self.add_noise()
        optimizer.step()
        optimizer.zero_grad(set_to_none=True)
        return n, c
