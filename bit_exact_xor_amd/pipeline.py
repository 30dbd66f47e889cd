"""Pipelined transfer of a stream through pinned host memory.

A pinned host buffer stands in for the network.  The sender runs
dcr_encode_pipelined and, while the encode is still going, copies each
slice it publishes device -> host on a stream of its own.  The receiver
copies each slice host -> its own device buffers on a second stream and
applies its records (dcr_apply with the slice's prefix header) on a third,
so the copy of slice k + 1 overlaps the apply of slice k.  Building and
sending overlap on the sender, receiving and patching on the receiver, and
the latency becomes about the longest leg rather than the sum (ai-feeds
summary "key modules" 5; humansand "weight teleportation" page,
"Overlapping DE and SM": the transfer into one slot runs while the bitwise
kernel works on the other).

Only copies (the copy engines) and library calls are issued here; every
step of the method runs in libdcr's kernels.

Fp4Refit is the same path for weights that the receiver serves in 4 bits:
the trainer's BF16 or fp32 weights are quantised, the bytes that changed
travel, and the receiver multiplies with the tensors the apply has patched.
"""
import contextlib

import numpy as np

from . import dcr


def _u64(h: np.ndarray, off: int) -> int:
    return int(h[off:off + 8].view("<u8")[0])


class HostLoopback:
    """Pinned host staging and the receiver's device copy of a stream."""

    def __init__(self, plan: "dcr.Plan", dir_bytes: int, payload_bytes: int, device="cuda"):
        import torch
        self.plan = plan
        self.host_dir = torch.empty(max(int(dir_bytes), 32), dtype=torch.uint8, pin_memory=True)
        self.host_payload = torch.empty(max(int(payload_bytes), 16), dtype=torch.uint8, pin_memory=True)
        self.rdir = torch.empty(self.host_dir.numel(), dtype=torch.uint8, device=device)
        self.rpayload = torch.empty(self.host_payload.numel(), dtype=torch.uint8, device=device)
        self.d2h = torch.cuda.Stream(device=device)
        self.h2d = torch.cuda.Stream(device=device)
        self.apply_stream = torch.cuda.Stream(device=device)
        self.device = device

    def _fits(self, r1, p1):
        if r1 > self.host_dir.numel() // 32 or p1 > self.host_payload.numel():
            raise dcr.DcrError(dcr.DCR_E_CAPACITY, "HostLoopback", "host staging smaller than the stream")

    # ------------------------------------------------------------ sender
    def send(self, old_shards, new_shards, mode, base_version, new_version, sb: "dcr.StreamBuffers", workspace,
             n_slices: int, timeout_us: int = 30_000_000):
        """Encode with a ready watermark on the current stream; copy each
        published slice to host memory as soon as it is published.  Returns
        the prefix headers and, per slice, an event that completes when the
        slice is in host memory."""
        import torch
        # kept on the object: after a failed wait the encode may still
        # publish into it, so it must not go back to torch's pinned pool
        self._ready = ready = torch.zeros(dcr.ready_region_bytes(n_slices), dtype=torch.uint8, pin_memory=True)
        dcr.dcr_encode_pipelined(self.plan, old_shards, new_shards, mode, base_version, new_version, sb.header,
                                 sb.dir, sb.payload, sb.result, workspace, n_slices, ready)
        n = int(ready.numpy()[12:16].view("<u4")[0])
        heads, sent = [], []
        r0 = p0 = 0
        for k in range(n):
            h = dcr.dcr_ready_wait(ready, k, timeout_us)
            r1, p1 = _u64(h, 40), _u64(h, 48)
            self._fits(r1, p1)
            with torch.cuda.stream(self.d2h):
                self.host_dir[r0 * 32:r1 * 32].copy_(sb.dir[r0 * 32:r1 * 32], non_blocking=True)
                self.host_payload[p0:p1].copy_(sb.payload[p0:p1], non_blocking=True)
                ev = torch.cuda.Event()
                ev.record(self.d2h)
            heads.append(h)
            sent.append(ev)
            r0, p0 = r1, p1
        return heads, sent

    def send_serial(self, old_shards, new_shards, mode, base_version, new_version, sb: "dcr.StreamBuffers",
                    workspace):
        """The sender without pipelining: the whole encode, then the whole
        stream device -> host.  Returns the header; the caller synchronises
        the device -> host stream."""
        import torch
        dcr.dcr_encode(self.plan, old_shards, new_shards, mode, base_version, new_version, sb.header, sb.dir,
                       sb.payload, sb.result, workspace)
        torch.cuda.current_stream().synchronize()      # the host needs the stream's size
        r = sb.result_host()
        if int(r["status"]) != 0:
            raise dcr.DcrError(int(r["status"]), "HostLoopback.send_serial", "encode failed")
        n, pb = int(r["n_records"]), int(r["payload_bytes"])
        self._fits(n, pb)
        with torch.cuda.stream(self.d2h):
            self.host_dir[:n * 32].copy_(sb.dir[:n * 32], non_blocking=True)
            self.host_payload[:pb].copy_(sb.payload[:pb], non_blocking=True)
        return sb.header_host()

    # ---------------------------------------------------------- receiver
    def receive(self, heads, canon, flags, apply_workspace, base_version, sent=None):
        """Copy each slice of a stream in host memory to the receiver's
        buffers and apply its records with its prefix header, the copy of a
        slice overlapping the apply of the one before.  `sent[k]` (optional)
        is an event the copy of slice k waits for.  Returns the apply results
        (device, one per slice with records); the caller synchronises the
        apply stream."""
        import torch
        results = []
        r0 = p0 = 0
        for k, h in enumerate(heads):
            r1, p1 = _u64(h, 40), _u64(h, 48)
            self._fits(r1, p1)
            if sent is not None:
                self.h2d.wait_event(sent[k])
            with torch.cuda.stream(self.h2d):
                self.rdir[r0 * 32:r1 * 32].copy_(self.host_dir[r0 * 32:r1 * 32], non_blocking=True)
                self.rpayload[p0:p1].copy_(self.host_payload[p0:p1], non_blocking=True)
                arrived = torch.cuda.Event()
                arrived.record(self.h2d)
            if r1 > r0:
                self.apply_stream.wait_event(arrived)
                with torch.cuda.stream(self.apply_stream):
                    res = torch.empty(32, dtype=torch.uint8, device=self.device)   # the apply initialises it
                    dcr.dcr_apply(self.plan, canon, h, self.rdir, self.rpayload, flags, r0, r1 - r0, base_version,
                                  res, apply_workspace, stream=self.apply_stream)
                results.append(res)
            r0, p0 = r1, p1
        return results

    def receive_serial(self, header, canon, flags, apply_workspace, base_version):
        """The receiver without pipelining: the whole stream host -> device,
        then one apply.  Returns the apply result; the caller synchronises
        the apply stream."""
        import torch
        n, pb = _u64(header, 40), _u64(header, 48)
        self._fits(n, pb)
        with torch.cuda.stream(self.h2d):
            self.rdir[:n * 32].copy_(self.host_dir[:n * 32], non_blocking=True)
            self.rpayload[:pb].copy_(self.host_payload[:pb], non_blocking=True)
        self.h2d.synchronize()
        with torch.cuda.stream(self.apply_stream):
            res = torch.empty(32, dtype=torch.uint8, device=self.device)
            dcr.dcr_apply(self.plan, canon, header, self.rdir, self.rpayload, flags, 0, n, base_version, res,
                          apply_workspace, stream=self.apply_stream)
        return res

    def receive_retry(self, header, canon, apply_workspace, base_version):
        """The receiver of a RETRY stream in host memory: the whole stream
        host -> device, then its overwrites, whatever an interrupted apply
        has already written.  Returns the apply result; the caller
        synchronises the apply stream."""
        import torch
        n, pb = _u64(header, 40), _u64(header, 48)
        self._fits(n, pb)
        with torch.cuda.stream(self.h2d):
            self.rdir[:n * 32].copy_(self.host_dir[:n * 32], non_blocking=True)
            self.rpayload[:pb].copy_(self.host_payload[:pb], non_blocking=True)
        self.h2d.synchronize()
        with torch.cuda.stream(self.apply_stream):
            res = torch.empty(32, dtype=torch.uint8, device=self.device)
            dcr.dcr_apply_overwrite_retry(self.plan, canon, header, self.rdir, self.rpayload, base_version, res,
                                          apply_workspace, stream=self.apply_stream)
        return res

    # ------------------------------------------------- both on one GPU
    def run(self, old_shards, new_shards, mode, base_version, new_version, sb: "dcr.StreamBuffers", workspace,
            n_slices: int, canon, flags, apply_workspace):
        """Sender and receiver together: each slice goes device -> host ->
        device and is applied while the encode and the later slices are
        still in flight.  Returns (prefix headers, apply results)."""
        heads, sent = self.send(old_shards, new_shards, mode, base_version, new_version, sb, workspace, n_slices)
        return heads, self.receive(heads, canon, flags, apply_workspace, base_version, sent)

    def run_serial(self, old_shards, new_shards, mode, base_version, new_version, sb: "dcr.StreamBuffers",
                   workspace, canon, flags, apply_workspace):
        """Both sides one step after the other."""
        h = self.send_serial(old_shards, new_shards, mode, base_version, new_version, sb, workspace)
        self.d2h.synchronize()
        return self.receive_serial(h, canon, flags, apply_workspace, base_version)


class Fp4Refit:
    """A refit of 4-bit weights over a HostLoopback.

    `shapes` lists the weights' (rows, cols).  The sender holds two versions of
    each as `Fp4Tensor`s, the committed one (`sent`) and the next; the receiver
    holds one (`held`), in memory of its own.  Codes and scale bytes are
    canonical tensors of one-byte elements carried as XOR masks, an NV tensor
    scale is one fp32 element carried as an overwrite.  The first refit takes
    the NV tensor scales from the weights and sends everything; later ones keep
    them (so that few bytes change) unless `calibrate` is passed.

    A refit that raises once it has begun to send may have patched part of
    `held` (`interrupted`): the masks must not be applied again, and products
    are refused.  recover() finishes it, the same change set as overwrites; so
    does the next refit before it starts.

    Calls come from one thread at a time, on any streams of the weights' GPU: a
    product reads the weights as the calls before it left them, and has scratch
    memory of its stream's own.  A refit waits for the streams that products
    were put on since the last one (which have to be there still).  Replays of
    a captured product are not seen here: a refit is called when they are
    done."""

    def __init__(self, shapes, fmt=dcr.FP4_NV, device="cuda", n_slices=4):
        import torch
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(device):
            self._make(shapes, fmt, device, n_slices)
            # (the first calls may come on other streams)
            torch.cuda.current_stream().synchronize()

    def _make(self, shapes, fmt, device, n_slices):
        import torch
        self.fmt, self.device, self.n_slices = fmt, device, n_slices
        self.version = 0
        self.interrupted = False
        self.products = {}               # streams with products since the last refit: (stream, scratch memory)
        self.sent, self.next, self.held = ([dcr.Fp4Tensor(r, c, fmt, device) for r, c in shapes] for _ in range(3))
        for side in (self.sent, self.next, self.held):
            for t in side:
                if t.tensor_scale is not None:
                    t.tensor_scale.zero_()
        sizes = []                       # (elements, bytes an element, route) of each canonical tensor
        for t in self.held:
            sizes += [(t.codes.numel(), 1, dcr.ROUTE_AFFINE_XOR), (t.scales.numel(), 1, dcr.ROUTE_AFFINE_XOR)]
            if fmt == dcr.FP4_NV:
                sizes.append((1, 4, dcr.ROUTE_OVERWRITE))
        tensors = np.zeros(len(sizes), dtype=dcr.TENSOR_DESC)
        segments = np.zeros(sum(n > 0 for n, _w, _r in sizes), dtype=dcr.SEGMENT)
        s = 0
        for i, (n, w, route) in enumerate(sizes):
            tensors[i] = (n, w, route, -1, 0)
            if n:                        # each tensor is its own shard, whole and in order
                segments[s] = (i, i, 1, 0, 0, 0, [n, 1, 1, 1], [1, 0, 0, 0], [1, 0, 0, 0])
                s += 1
        self.plan = dcr.dcr_plan_build(tensors, [n * w for n, w, _r in sizes], segments)
        dcr.dcr_plan_upload(self.plan, device)
        info = self.plan.info
        self.link = HostLoopback(self.plan, info.max_dir_bytes, info.max_payload_bytes, device)
        self.stream = dcr.StreamBuffers(self.plan, device)
        self.flags = torch.empty(max(1, info.max_dir_bytes // 32), dtype=torch.uint8, device=device)
        self.encode_workspace = dcr.workspace(self.plan, device, info.max_payload_bytes)
        self.apply_workspace = dcr.workspace(self.plan, device)
        self.fp4_workspace = dcr.fp4_workspace(device)

    def _buffers(self, side):
        out = []
        for t in side:
            out += [t.codes, t.scales]
            if t.tensor_scale is not None:
                out.append(t.tensor_scale)
        return out

    def refit(self, weights, calibrate=False):
        """Quantise the trainer's `weights` (BF16 or fp32, one for each shape),
        send what changed and patch `held`; returns the payload bytes sent.
        The work runs on the current stream and the link's; `held` is patched
        when the call returns."""
        if len(weights) != len(self.next):
            raise ValueError(f"{len(self.next)} weights expected, got {len(weights)}")
        self.recover()
        calibrate = self.fmt == dcr.FP4_NV and (calibrate or self.version == 0)
        with self._drained():
            for w, q, old in zip(weights, self.next, self.sent):
                if q.tensor_scale is not None and not calibrate:
                    q.tensor_scale.copy_(old.tensor_scale)
                dcr.dcr_fp4_quantize(w, q, dcr.FP4_CALIBRATE if calibrate else 0, self.fp4_workspace)
            self.flags.zero_()
            self._before_applies()           # (the flags, too)
            self.interrupted = True          # until all of it has arrived
            heads, results = self.link.run(self._buffers(self.sent), self._buffers(self.next), dcr.MODE_DELTA,
                                           self.version, self.version + 1, self.stream, self.encode_workspace,
                                           self.n_slices, self._buffers(self.held), self.flags, self.apply_workspace)
            self._arrived(results)
        return _u64(heads[-1], 48)

    def recover(self):
        """Finish an interrupted refit: the bytes that it changes, sent again
        as overwrites (idempotent, so what its applies have done does not
        matter).  Nothing is done where none was interrupted."""
        if not self.interrupted:
            return
        with self._drained():
            header = self.link.send_serial(self._buffers(self.sent), self._buffers(self.next), dcr.MODE_RETRY,
                                           self.version, self.version + 1, self.stream, self.encode_workspace)
            self.link.d2h.synchronize()
            self._before_applies()
            self._arrived([self.link.receive_retry(header, self._buffers(self.held), self.apply_workspace,
                                                   self.version)])

    @contextlib.contextmanager
    def _drained(self):
        """On the weights' GPU and its current stream; an error leaves when
        nothing is in flight: the next call, on whatever stream, uses the same
        buffers."""
        import torch
        with torch.cuda.device(self.device):
            try:
                yield
            except BaseException:
                for s in (torch.cuda.current_stream(), self.link.d2h, self.link.h2d, self.link.apply_stream):
                    s.synchronize()
                raise

    def _before_applies(self):
        """The receiver's streams wait for what the current one holds and for
        the products of all."""
        import torch
        for stream in (torch.cuda.current_stream(), *(s for s, _workspace in self.products.values())):
            self.link.apply_stream.wait_stream(stream)

    def _arrived(self, results):
        """Wait for the applies of a stream; with all of it in `held`, the
        next version is the sent one."""
        self.link.apply_stream.synchronize()
        for r in results:
            bad = dcr.apply_result(r)
            if int(bad["n_invalid"]):
                raise dcr.DcrError(dcr.DCR_E_FORMAT, "Fp4Refit", f"{int(bad['n_invalid'])} records refused")
        self.sent, self.next, self.version, self.interrupted = self.next, self.sent, self.version + 1, False
        self.products.clear()

    def matmul(self, i, x, out_dtype=None, offsets=None, y=None):
        """x w^T with the receiver's weight i (see dcr_fp4_matmul), in a new
        tensor or in `y`.  With `offsets`, rows of x in front of the first
        group and behind the last give zeros, and leave those of `y` as they
        are."""
        import torch
        if self.interrupted:
            raise dcr.DcrError(dcr.DCR_E_VERSION, "Fp4Refit.matmul", "the last refit was interrupted: recover() first")
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self.matmul(i, x, out_dtype, offsets, y)
        w = self.held[i]
        if y is None:
            _off, _g, n = dcr._groups(w, offsets)
            make = torch.empty if offsets is None else torch.zeros
            y = make(x.shape[0], n, dtype=out_dtype or x.dtype, device=x.device)
        if torch.cuda.is_current_stream_capturing():
            workspace = dcr.fp4_workspace(self.device)       # (of the graph's memory)
        else:
            raw = torch._C._cuda_getCurrentRawStream(self.device.index)
            if raw not in self.products:
                self.products[raw] = (torch.cuda.current_stream(), dcr.fp4_workspace(self.device))
            workspace = self.products[raw][1]
        dcr.dcr_fp4_matmul(x, w, y, offsets, workspace)
        return y
