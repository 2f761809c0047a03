"""The device workspace that a plan or an operator object owns, and the streams
that use it."""

from __future__ import annotations

from typing import Optional

from . import _lib as L


def stream_of(handle: int, dev: int):
    """The torch stream of a raw handle on device `dev` (0 is the default stream)."""
    import torch
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


def _capturing(stream) -> bool:
    import torch
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


class Workspace:
    """Mixin: the workspace tensor, its status word and the streams that use it.

    The tensor comes from the caching allocator on the device's current stream.
    Every other stream that a call uses first waits until the workspace is
    cleared and is recorded with the allocator, so that the memory is not handed
    out again before the calls on it are done, even if the object is dropped
    right after run(). A raw stream has to outlive the object. Replays of a graph
    that captured a call use the workspace too, unseen by the allocator: keep the
    object as long as the graph."""

    workspace = None
    workspace_bytes = 1024
    _at = -1, 0          # the workspace's device and address
    _streams = ()        # raw handles that wait for the clearing and are recorded
    _cleared = None      # event behind the clearing
    _allocates_under_capture = False   # a first run may take its workspace from a graph's own memory

    def allocate_workspace(self, device, stream: Optional[int] = None):
        """Allocates and clears the workspace on `stream` (default: the device's current stream)."""
        import torch
        with torch.cuda.device(torch.device(device)):
            dev = torch.cuda.current_device()
            current = torch.cuda.current_stream()
            on = current if stream is None or stream == current.cuda_stream else stream_of(stream, dev)
            if on is not current:
                if _capturing(on):
                    raise RuntimeError("allocate_workspace() before capturing")
                on.wait_stream(current)   # the memory may have been used there
            workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device="cuda")
            if on is not current:
                workspace.record_stream(on)
            L.mla_workspace_init(workspace.data_ptr(), self.workspace_bytes, on.cuda_stream)
            cleared = None
            if not torch.cuda.is_current_stream_capturing():
                cleared = torch.cuda.Event()
                cleared.record(on)
        self.workspace, self._cleared = workspace, cleared
        self._at = dev, workspace.data_ptr()
        self._streams = {on.cuda_stream}
        return self

    def _stream(self, dev: int, stream: Optional[int]) -> int:
        """The raw stream of a call on device `dev` (default: its current stream), ready to use the workspace, which is
        allocated if there is none yet."""
        import torch
        if self.workspace is None:
            with torch.cuda.device(dev):
                capturing = torch.cuda.is_current_stream_capturing() or (
                    stream is not None and _capturing(stream_of(stream, dev)))
            if capturing and not self._allocates_under_capture:
                raise RuntimeError("allocate_workspace() before capturing: memory allocated under a capture belongs "
                                   "to the graph")
            self.allocate_workspace(dev, None if capturing else stream)
        if self._at[0] != dev:
            raise ValueError(f"the workspace is on device {self._at[0]}, the tensors on device {dev}")
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(dev)   # torch.cuda.current_stream(dev) costs a microsecond more
        if stream not in self._streams:
            s = stream_of(stream, dev)
            if not _capturing(s):   # captured work runs when the graph does
                if self._cleared is not None:
                    s.wait_event(self._cleared)
                self.workspace.record_stream(s)
                self._streams.add(stream)
        return stream

    def read_status(self, stream: Optional[int] = None) -> int:
        """The first error that the device recorded since the last call (an mla_status_t), cleared. Synchronises `stream`
        (default: the device's current stream): give the stream that the calls ran on."""
        import torch
        if self.workspace is None:
            return L.MLA_OK     # nothing has run
        with torch.cuda.device(self.workspace.device):
            if stream is None:
                stream = torch.cuda.current_stream().cuda_stream
            return L.mla_decode_read_status(self.workspace.data_ptr(), stream)
