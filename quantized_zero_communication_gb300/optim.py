"""AdamW over the tensors of a parameter shard: fp32 master weights, states in fp32 or in
8 bits, one library call per step (``zpp_adamw_step_counted``), which also takes the gradient norm
when it clips; and Muon (``zpp_muon_step``) for whole matrices. Everything stays on the device; a
step never synchronises.

The 16-bit tensors in ``weights`` receive the updated parameters, ready for the next
all-gather's ``quant_blockwise``.
"""
import array
import ctypes
import math

from . import binding as _b


class AdamW:
    """AdamW (decoupled weight decay) over a list of at most 1024 contiguous fp32 CUDA tensors (or a
    single one, here and wherever a list is named).

    state_bits 32 holds both states in fp32; 8 holds m and sqrt(v) as float8_e4m3fn codes
    with one fp32 scale per 256 elements, rounded stochastically from `seed` and the step
    (see include/zpp.h). weights: fp16 or bf16 tensors of the parameters' sizes that each
    step fills, or None. exp_avg, exp_avg_sq, scales and step resume from a saved state()
    (the tensors are taken over, not copied); by default the states start at zero. An optimiser is
    made and stepped on one stream, or on streams that wait for each other.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, *,
                 state_bits=32, weights=None, seed=0, exp_avg=None, exp_avg_sq=None, scales=None,
                 step=0):
        torch = _b._torch()
        f32 = (_b.ZPP_F32,)
        as_list = lambda ts: [ts] if isinstance(ts, torch.Tensor) else list(ts)  # noqa: E731
        self.params = as_list(params)
        if not self.params:
            raise ValueError("AdamW needs at least one tensor")
        if len(self.params) > _b.ZPP_MAX_TENSORS:
            raise ValueError(f"AdamW: {len(self.params)} tensors, at most {_b.ZPP_MAX_TENSORS} to a call: "
                             "flatten them, or take an optimiser for each part")
        if state_bits not in (8, 32):
            raise ValueError("state_bits: 8 or 32")
        if (exp_avg is None) != (exp_avg_sq is None):
            raise ValueError("exp_avg and exp_avg_sq come together")
        if (scales is not None) != (state_bits == 8 and exp_avg is not None):
            raise ValueError("scales come with exp_avg and exp_avg_sq of state_bits 8")
        if not 0 <= seed < 1 << 32:
            raise ValueError("seed: 0 .. 2^32 - 1")
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits, self.seed = state_bits, seed
        self._sizes = array.array("q", [p.numel() for p in self.params])
        self._blocks = _b._state_blocks(self._sizes)
        code = torch.float32 if state_bits == 32 else torch.float8_e4m3fn

        def states(given, sizes, dtype):
            if given is not None:
                return as_list(given)
            # one buffer, every tensor's part 256 elements aligned
            at, end = [], 0
            for n in sizes:
                at.append(end)
                end += -(-n // 256) * 256
            # (as bytes: zero is all bits zero in both types)
            flat = torch.zeros(end * dtype.itemsize, dtype=torch.uint8,
                               device=self.params[0].device).view(dtype)
            return [flat[o:o + n] for o, n in zip(at, sizes)]

        self.exp_avg = states(exp_avg, self._sizes, code)
        self.exp_avg_sq = states(exp_avg_sq, self._sizes, code)
        self.scales = None
        if state_bits == 8:
            self.scales = tuple(states(s, self._blocks, torch.float32)
                                for s in (scales or (None, None)))
        self.weights = None if weights is None else as_list(weights)
        state = f32 if state_bits == 32 else (_b._E4M3,)
        self._lists = [("params", 0, self.params, self._sizes, f32),
                       ("exp_avg", 2, self.exp_avg, self._sizes, state),
                       ("exp_avg_sq", 3, self.exp_avg_sq, self._sizes, state)]
        if state_bits == 8:
            self._lists += [(f"scales[{k}]", 4 + k, self.scales[k], self._blocks, f32)
                            for k in (0, 1)]
        if self.weights is not None:
            self._lists.append(("weights", 6, self.weights, self._sizes,
                                (_b.ZPP_F16, _b.ZPP_BF16)))
        self._device = None
        self._table = array.array("q", bytes(64 * len(self.params)))
        self._table[7::8] = self._sizes
        self._hp = _b.AdamwParams(lr, *self.betas, eps, weight_decay, step, seed)
        self._work = _b.zpp_grad_norm_workspace(sum(self._sizes), len(self._sizes))
        self._w_kind = _b.ZPP_BF16
        self._gather()
        # The number of the last step on the device (zpp_adamw_record), and here as long as no step
        # may have been skipped: _known is None afterwards.
        self._record = torch.zeros(8, dtype=torch.int64, device=self.params[0].device)
        if step:
            self._record[:1].fill_(step)
        self._known = step

    @property
    def steps(self):
        """The steps taken; skipped ones do not count. Once a step was clipped or scaled only the
        device knows, and reading this waits for it. Setting it gives the next step's number, less
        one."""
        return self._known if self._known is not None else int(self._record[0])

    @steps.setter
    def steps(self, step):
        self._record.zero_()
        self._record[:1].fill_(step)
        self._known = None

    def _enter(self, name, column, tensors, sizes, kinds):
        """Checks a list and writes its addresses into the call's table; their dtype's kind."""
        if len(tensors) != len(sizes):
            raise ValueError(f"{name}: {len(tensors)} tensors, expected {len(sizes)}")
        kind, device, same = _b._tensors().enter(tensors, self._table, column, sizes)
        if kind not in kinds or device < 0 or not same:
            _b._same_sizes(name, _b._dev_list(tensors, name, kinds)[1], sizes)
        if self._device is None:
            self._device = device
        if device != self._device:
            raise ValueError("all tensors of a call must be on one device")
        return kind

    def _gather(self):
        """Every tensor that the optimiser holds, as it is now (storage may have moved)."""
        for entry in self._lists:
            kind = self._enter(*entry)
            if entry[0] == "weights":
                self._w_kind = kind

    def step(self, grads, *, max_norm=None, pre_scale=None, grad_scale=None, lr=None):
        """One step with `grads` (contiguous, one of fp16 / bf16 / fp32, in the parameters'
        order). max_norm and / or pre_scale: the gradients are multiplied by pre_scale (say 1 /
        loss scale) and clipped to max_norm, the norm of these gradients together, and fp32 [2]
        (norm, factor) is returned; a norm that is not finite leaves parameters, states and the count
        of steps as they were. grad_scale: instead, an fp32 device tensor whose first element
        multiplies the gradients. A rank that owns a slice of a model needs that form: the factor
        has to be the same on all ranks, so their norms' squares are added up first (an
        all-reduce), and a total that is not finite has to give NaN:

            square = zpp.grad_norm(grads)[0].square()
            torch.distributed.all_reduce(square)
            total = square.sqrt()
            factor = torch.where(total.isfinite(), (max_norm / total).clamp(max=1.0), math.nan)
            opt.step(grads, grad_scale=factor.reshape(1))

        lr replaces the optimiser's for this step and the following ones."""
        torch = _b._torch()
        grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
        self._gather()
        kind = self._enter("grads", 1, grads, self._sizes, _b._GRAD_KINDS)
        if lr is not None:
            self.lr = lr
        scale, clip = 0, None
        if max_norm is not None or pre_scale is not None:
            if grad_scale is not None:
                raise ValueError("grad_scale replaces max_norm and pre_scale")
            clip = (math.inf if max_norm is None else max_norm,
                    1.0 if pre_scale is None else pre_scale, self._work)
        elif grad_scale is not None:
            scale = _b._scale_address(grads[0], grad_scale)
        hp = self._hp
        hp.lr, hp.step = self.lr, 0 if self._known is None else self._known + 1
        hp.beta1, hp.beta2 = self.betas
        hp.eps, hp.weight_decay = self.eps, self.weight_decay
        args = (_b._address("zpp_adamw_step_counted"), self._table, kind, self._w_kind, self.state_bits,
                ctypes.addressof(hp), scale, clip, self._record.data_ptr(), self._device)
        norm = _b._tensors().step(*args)
        if norm is False:  # another device is current
            with torch.cuda.device(self._device):
                norm = _b._tensors().step(*args)
        if type(norm) is int:
            raise _b.ZppError(norm, "zpp_adamw_step_counted")
        # (in a captured stream hp.step is 0 now: a replay is another step, the device counts them)
        self._known = None if clip or scale or not hp.step else hp.step
        return norm

    def state(self):
        """What a checkpoint keeps, as the constructor takes it: the state tensors themselves
        and the step count (which waits for the device once a step was clipped or scaled)."""
        return dict(exp_avg=self.exp_avg, exp_avg_sq=self.exp_avg_sq, scales=self.scales,
                    step=self.steps, seed=self.seed, state_bits=self.state_bits)


_ADJUST = ("original", "match_rms_adamw", "none")


class Muon:
    """Muon over a list of at most 1024 contiguous fp32 CUDA matrices (or a single one): momentum, an
    update made nearly orthogonal by Newton-Schulz steps, decoupled weight decay. It wants whole
    matrices, not slices of a flat shard; vectors and embeddings go to AdamW.

        m = momentum m + (1 - momentum) g,  u = (1 - momentum) g + momentum m  (nesterov; else m)
        p = p (1 - lr weight_decay) - lr adj orthogonalize(u, steps, coefficients, eps)

    adjust: "original": adj = sqrt(max(1, rows / cols)); "match_rms_adamw": 0.2 sqrt(max(rows, cols)),
    with which AdamW's lr and weight_decay do; "none": 1. weights: fp16 or bf16 matrices of the
    parameters' shapes that each step fills, or None. buffers: the momenta of a saved state() (taken over,
    not copied); by default they start at zero. An optimiser is made and stepped on one stream, or on
    streams that wait for each other.
    """

    def __init__(self, params, lr=1e-3, momentum=0.95, weight_decay=0.1, *, nesterov=True, steps=5,
                 coefficients=_b.NS_COEFFICIENTS, eps=1e-7, adjust="original", weights=None,
                 buffers=None):
        torch = _b._torch()
        as_list = lambda ts: [ts] if isinstance(ts, torch.Tensor) else list(ts)  # noqa: E731
        self.params = as_list(params)
        if not self.params:
            raise ValueError("Muon needs at least one matrix")
        if len(self.params) > _b.ZPP_MAX_TENSORS:
            raise ValueError(f"Muon: {len(self.params)} matrices, at most {_b.ZPP_MAX_TENSORS} to a call: "
                             "take an optimiser for each part")
        if adjust not in _ADJUST:
            raise ValueError(f"adjust: one of {_ADJUST}")
        _b._sides(self.params, "params")
        self._ns, self._coefficients = _b._steps(steps, coefficients, eps)
        self.lr, self.momentum, self.weight_decay = lr, momentum, weight_decay
        self.nesterov, self.adjust = nesterov, adjust
        self._shapes = [tuple(p.shape) for p in self.params]
        f32 = (_b.ZPP_F32,)
        _b._dev_list(self.params, "params", f32)
        self.buffers = ([torch.zeros_like(p) for p in self.params] if buffers is None
                        else as_list(buffers))
        self.weights = None if weights is None else as_list(weights)
        self._table = (_b.MuonTensor * len(self.params))()
        for row, (rows, cols) in zip(self._table, self._shapes):
            row.rows, row.cols = rows, cols
        self._lists = [("params", "param", self.params, f32), ("buffers", "momentum", self.buffers, f32)]
        if self.weights is not None:
            self._lists.append(("weights", "weight", self.weights, (_b.ZPP_F16, _b.ZPP_BF16)))
        self._device, self._w_kind = None, _b.ZPP_BF16
        self._gather()
        self._work = int(_b.lib().zpp_muon_workspace(ctypes.addressof(self._table), len(self._table)))

    def _enter(self, name, field, tensors, kinds):
        """Checks a list and writes its addresses into the call's table; their dtype's kind."""
        if len(tensors) != len(self._shapes):
            raise ValueError(f"{name}: {len(tensors)} matrices, expected {len(self._shapes)}")
        for i, (t, shape) in enumerate(zip(tensors, self._shapes)):
            if tuple(t.shape) != shape:
                raise ValueError(f"{name}[{i}]: {tuple(t.shape)}, expected {shape}")
        ptrs, _, kind, device = _b._dev_list(tensors, name, kinds)
        if self._device is None:
            self._device = device
        if device != self._device:
            raise ValueError("all tensors of a call must be on one device")
        for row, p in zip(self._table, ptrs):
            setattr(row, field, p)
        return kind

    def _gather(self):
        """Every tensor that the optimiser holds, as it is now (storage may have moved)."""
        for name, field, tensors, kinds in self._lists:
            kind = self._enter(name, field, tensors, kinds)
            if name == "weights":
                self._w_kind = kind

    def step(self, grads, *, max_norm=None, pre_scale=None, grad_scale=None, lr=None):
        """One step with `grads` (contiguous, one of fp16 / bf16 / fp32, in the parameters' order and
        shapes). max_norm, pre_scale, grad_scale and what is returned: as AdamW.step; a factor that is
        not finite leaves parameters, weights and momenta as they were. (The direction of an update
        does not depend on the gradients' scale, but what they weigh in the momentum does.) lr replaces
        the optimiser's for this step and the following ones. A graph that kept a parameter's, weight's or
        momentum's values of before the step raises in its backward pass."""
        torch = _b._torch()
        grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
        self._gather()
        kind = self._enter("grads", "grad", grads, _b._GRAD_KINDS)
        if lr is not None:
            self.lr = lr
        norm, scale = None, 0
        if max_norm is not None or pre_scale is not None:
            if grad_scale is not None:
                raise ValueError("grad_scale replaces max_norm and pre_scale")
            # (matrices may start anywhere, the norm's tensors at multiples of 16 bytes: others are copied)
            norm = _b.grad_norm([g if g.data_ptr() % 16 == 0 else g.clone() for g in grads], max_norm,
                                1.0 if pre_scale is None else pre_scale)
            scale = norm.data_ptr() + 4
        elif grad_scale is not None:
            scale = _b._scale_address(grads[0], grad_scale)
        hp = _b.MuonParams(self.lr, self.momentum, self.weight_decay, bool(self.nesterov),
                           _ADJUST.index(self.adjust), self._ns)
        work = torch.empty(max(self._work, 0), dtype=torch.uint8, device=self.params[0].device)
        _b._launch(self._device, "zpp_muon_step", ctypes.addressof(self._table), len(self._table), kind,
                   self._w_kind, ctypes.addressof(hp), scale, work.data_ptr())
        _b._written(*self.params, *self.buffers, *(self.weights or ()))
        return norm

    def state(self):
        """What a checkpoint keeps, as the constructor takes it: the momenta themselves."""
        return dict(buffers=self.buffers)
